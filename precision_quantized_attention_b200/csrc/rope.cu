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
#include <type_traits>

#include "launch.h"
#include "quant_math.cuh"
#include "sm100_ptx.cuh"

namespace qattn {

// -------------------------------------------------------------------------------------------
// Rotary table.  The angle of a far position needs more than 32 bits before it is reduced, and a small sine, of a small
// angle or next to a multiple of pi, needs the bits behind the first 32 of its turn.  So the turn is held in 64 bits, in
// fixed point, where the reduction to one turn is the overflow of the words: position (32.64 bits) times the pair's
// frequency in turns, 64 bits of fraction.  The nearest quarter turn and a rest of at most an eighth follow; cos and sin of
// the rest, rounded to 24 bits, are FP32 sums: 6 x 2^-24 of their value.  (With the turn cut off at 32 bits a sine near
// 1e-6 was off by 6e-4 of itself.)  118800 tokens of 64 pairs: 13.9 us, 4.5 TB/s, bound by the integer and FP32
// instructions; with fractional positions, whose products are two more, 17.5 us; 4608 tokens 2.4 us, a launch.  With the product and the reduction in FP64 (four operations and
// a conversion a pair) the FP64 path bounded the kernel: 118800 tokens of 64 pairs took 21 us.
// A block takes 32 to 128 tokens, as many as fill whole rounds of resident blocks: their positions are split into words
// once, then a thread keeps one pair, its frequency in registers, and steps over the tokens; a block's stores are
// contiguous.
// -------------------------------------------------------------------------------------------
constexpr int TABLE_TOKENS = 128;
constexpr int TABLE_BLOCKS = 6;                    // resident on an SM

// A position as magnitude and sign: |position| = ip + (f_hi + f_lo / 2^32) / 2^32.
struct alignas(16) TablePosInt {
  uint32_t ip, sign;                               // sign: the sine's sign bit
  float off;                                       // 2^-30; NaN for a position that is not finite or past 2^31
};
struct alignas(8) TablePosFloat {
  uint32_t ip, sign;
  float off;
  uint32_t f_hi, f_lo;
};

__device__ __forceinline__ TablePosInt split_position(int v) {
  const uint32_t u = static_cast<uint32_t>(v);
  return {v < 0 ? 0u - u : u, u & 0x80000000u, 0x1p-30f};
}
// Every step is exact: a float has 24 bits, so what is left of one below 1 or below 2^-32 is a float too.
__device__ __forceinline__ TablePosFloat split_position(float v) {
  if (!(v >= -2147483648.0f && v < 2147483648.0f)) return {0u, 0u, __int_as_float(0x7FFFFFFF), 0u, 0u};
  const float m = fabsf(v);
  const uint32_t ip = __float2uint_rz(m);
  const float f = (m - static_cast<float>(ip)) * 4294967296.0f;
  const uint32_t f_hi = __float2uint_rz(f);
  return {ip, __float_as_uint(v) & 0x80000000u, 0x1p-30f, f_hi,
          __float2uint_rz((f - static_cast<float>(f_hi)) * 4294967296.0f)};
}

// What the fraction adds to the phase: the products' bits from 2^-64 on.
__device__ __forceinline__ uint64_t fraction_phase(const TablePosInt&, uint32_t, uint32_t) { return 0; }
__device__ __forceinline__ uint64_t fraction_phase(const TablePosFloat& v, uint32_t hi, uint32_t lo) {
  return static_cast<uint64_t>(v.f_hi) * hi + __umulhi(v.f_hi, lo) + __umulhi(v.f_lo, hi);
}
__device__ __forceinline__ uint32_t has_fraction(const TablePosInt&) { return 0; }
__device__ __forceinline__ uint32_t has_fraction(const TablePosFloat& v) { return v.f_hi | v.f_lo; }

template <class P>
__global__ void __launch_bounds__(256, TABLE_BLOCKS) k_rope_table(const P* __restrict__ pos, int64_t pos_stride, int tokens,
                                                    int per_block, int axes, const __grid_constant__ RopeFreqs f,
                                                    float2* __restrict__ table, int* __restrict__ err) {
  // block: x = pair, y = token within a pass (no division)
  using Pos = decltype(split_position(P()));
  __shared__ Pos at[TABLE_TOKENS * 8];             // 8 = most axes
  const int pairs = blockDim.x, p = threadIdx.x;
  const int t0 = static_cast<int>(blockIdx.x) * per_block;
  const int n = min(per_block, tokens - t0);
  uint32_t fraction = 0;
  for (int t = threadIdx.y * pairs + p; t < n; t += pairs * blockDim.y)
    for (int a = 0; a < axes; ++a) {
      const Pos v = split_position(__ldg(pos + (t0 + t) * pos_stride + a));
      fraction |= has_fraction(v);
      at[t * 8 + a] = v;
    }
  if constexpr (std::is_same_v<P, float>) fraction = __syncthreads_or(static_cast<int>(fraction));
  else __syncthreads();
  // Through a generic address: indexed by the thread, the constant bank serves one lane at a time (10 us of the 118800
  // tokens above).
  const RopeFreqs* freqs = &f;
  asm volatile("" : "+l"(freqs));
  const RopePair mine_f = freqs->pair[p];
  const uint32_t hi = static_cast<uint32_t>(mine_f.turns >> 32), lo = static_cast<uint32_t>(mine_f.turns);
  const Pos* mine = at + mine_f.axis;
  float2* out = table + static_cast<int64_t>(t0) * pairs + p;
  auto entries = [&](auto fractions) {
#pragma unroll 4
    for (int t = threadIdx.y; t < n; t += blockDim.y) {
      const Pos v = mine[t * 8];
      uint64_t phase = mine_f.turns * v.ip;          // the turn's 64 bits
      if constexpr (decltype(fractions)::value) phase += fraction_phase(v, hi, lo);
      const uint32_t ph = static_cast<uint32_t>(phase >> 32);
      const uint32_t q = (ph + 0x20000000u) >> 30;             // nearest quarter turn
      // The rest x, |x| <= 1/2 quarter turns: its high word in units of 2^-30, and the low word's first 23 bits behind it
      // (the mantissa of a float in [2^-30, 2^-29)), so that a small sine keeps 24 bits.  Then Taylor sums of
      // sin(pi x / 2) / x and cos(pi x / 2) in x^2: coefficients (pi / 2)^k / k!, the first ones left out below 2^-28
      const float low = __uint_as_float((static_cast<uint32_t>(phase) >> 9) + 0x30800000u) - v.off;
      const float x = fmaf(static_cast<float>(static_cast<int>(ph - (q << 30))), 0x1p-30f, low), z = x * x;
      const float s =
          x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 0.0001604411848f, -0.004681754135f), 0.07969262625f), -0.6459640975f), 1.570796327f);
      const float c =
          fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.520204237e-05f, 0.0009192602748f), -0.02086348076f), 0.2536695079f), -1.23370055f), 1.0f);
      // a quarter turn swaps them and negates the new cosine, half a turn negates both, a negative position the sine
      const uint32_t flip = (q & 2u) << 30;
      const float c1 = (q & 1u) ? -s : c, s1 = (q & 1u) ? c : s;
      if (QATTN_IN_BOUNDS(err, t0 + t < tokens && p < pairs))
        out[t * pairs] =
            make_float2(__uint_as_float(__float_as_uint(c1) ^ flip), __uint_as_float(__float_as_uint(s1) ^ flip ^ v.sign));
    }
  };
  // a block of whole numbers leaves the fractions' products out
  if (fraction != 0) entries(std::true_type{});
  else entries(std::false_type{});
}

cudaError_t launch_rope_table(const void* pos, int pos_is_float, int64_t pos_stride, int tokens, int axes,
                              int pairs, const RopeFreqs& f, float* table, int* err, int num_sms,
                              cudaStream_t stream) {
  const int64_t round = static_cast<int64_t>(num_sms) * TABLE_BLOCKS;
  const int64_t rounds = (tokens - 1) / (round * TABLE_TOKENS) + 1;
  int per_block = static_cast<int>((tokens - 1) / (round * rounds) + 1);
  if (per_block < 32) per_block = 32;
  const unsigned grid = static_cast<unsigned>((tokens - 1) / per_block + 1);
  const dim3 block(static_cast<unsigned>(pairs), static_cast<unsigned>(256 / pairs));
  if (pos_is_float)
    k_rope_table<float><<<grid, block, 0, stream>>>(static_cast<const float*>(pos), pos_stride, tokens, per_block,
                                                    axes, f, reinterpret_cast<float2*>(table), err);
  else
    k_rope_table<int><<<grid, block, 0, stream>>>(static_cast<const int*>(pos), pos_stride, tokens, per_block,
                                                  axes, f, reinterpret_cast<float2*>(table), err);
  return cudaGetLastError();
}

// -------------------------------------------------------------------------------------------
// Norm + rotation.  A head row of D channels is held by a group of G lanes, two chunks of eight
// channels (16-byte loads) a lane, chunks gl and gl + ceil(D / 16), so a warp works on 32 / G heads at once
// and the sum of squares is a shuffle over the group.  A warp takes one token and a run of its heads: the
// token's cos and sin times the norm's weights are formed once as two coefficients a channel,
//   y_j = r * (a_j x_j + b_j x_partner(j)),   a = w cos,   b = -/+ w_partner sin,
// and reused for every head.  (A warp with more groups than the tensor has heads takes several tokens.)
// Statistics, coefficients and products are 32-bit; y is rounded once, to the tensor's 16-bit type or, with
// E4M3's 1 / scale in r, to its code.  Without norm and rotation (V) the codes are
// qattn_quantize_fp8's, the quotient correctly rounded.
//
// Bound by memory if the instructions fit: at 6.5 TB/s an SM has 23 ns, 170 issue slots, for 64 elements in and out as
// E4M3.  So the arithmetic runs on packed pairs of floats, a lane holds sixteen channels (with eight, the address,
// shuffle and rsqrt work counted twice as much), loads wait in shared memory and not in registers, and bodies without a
// branch inside are made for 16-bit and E4M3 output, with and without arithmetic: 22 instructions an element became 12.
// 8704 tokens x 24 heads x 128, Q, K and V: E4M3 43.3 us (5.7 TB/s, 0.86 of the copy bandwidth; 65 % of the issue
// slots), 4608 tokens bf16 29.3 us (5.9 TB/s, 0.90).
//
// With adjacent channels as partners (ROT_PAIRS) a packed pair holds the first channels of two partner
// pairs, another their second channels, so that no half has to be swapped.  With halves as partners and the
// whole head rotated (ROT_HALVES) the partner chunk is the lane's other chunk; a partial rotation
// (ROT_SHUFFLE) fetches it from its lane, from the first chunks only where no other is rotated (ROT_LOW).  A channel that is
// not rotated has no partner: the product with one would be 0 * infinity where the row holds an infinity.  ROT_PAIRS_PART
// leaves it out (8704 tokens, 96 of 128 channels rotated, E4M3: 46.0 us, 43.8 with the product; in ROT_PAIRS and ROT_HALVES
// every channel is rotated, at no such cost); in the shuffled modes the channel is its own
// partner, each with half of the weight.
// -------------------------------------------------------------------------------------------
enum { ROT_PAIRS = 0, ROT_HALVES = 1, ROT_SHUFFLE = 2, ROT_LOW = 3, ROT_PAIRS_PART = 4 };
__host__ __device__ constexpr bool adjacent(int mode) { return mode == ROT_PAIRS || mode == ROT_PAIRS_PART; }

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

// acc + 0 * w in the 16-bit type: stays 0 as long as every w is finite, NaN after.
template <bool FP16>
__device__ __forceinline__ uint32_t note_nonfinite(uint32_t w, uint32_t acc) {
  uint32_t d;
  if (FP16) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
  else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
  return d;
}

// Scale of E4M3 codes: s, and for the fast quotient (r, r) = RN(1 / s) and (-s, -s).
struct CodeDiv {
  float s;
  bool fast;
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

// Four warps a block and five blocks an SM (96 registers): 8704 tokens as E4M3 49 us then, with 8 warps x 2 or 3 blocks
// 56 and 53, 6 blocks (spills) 51; two warps x 10 blocks the same.
constexpr int ROPE_WARPS = 4, ROPE_BLOCKS = 5;
// Steps whose loads are in flight: they go to shared memory (cp.async, each lane to its own words, so that no barrier
// is needed), which leaves the registers to the arithmetic.
// A depth of 3 and 4 measured the same, 5 and 8 slower.
constexpr int ROPE_DEPTH = 3;
constexpr int ROPE_STEP_BYTES = 32 * 2 * 16;       // a warp's step: two chunks a lane
constexpr int ROPE_SMEM = ROPE_WARPS * (ROPE_DEPTH + 1) * ROPE_STEP_BYTES;

// 16 bytes to shared memory, zeros without a read where !valid.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Eight floats (two 16-byte loads).
__device__ __forceinline__ void load_f8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Channels (j0, j1) of a chunk that packed pair i holds.
template <int MODE>
__device__ __forceinline__ constexpr int pair_lo(int i) {
  return adjacent(MODE) ? (i < 2 ? 4 * i : 4 * (i - 2) + 1) : 2 * i;
}
template <int MODE>
__device__ __forceinline__ constexpr int pair_hi(int i) {
  return adjacent(MODE) ? pair_lo<MODE>(i) + 2 : pair_lo<MODE>(i) + 1;
}

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

// Coefficients of one chunk (channels c0 ..) of a token: the weight alone where nothing is rotated.  There b is
// 0, unless the chunk's partner is then itself (SELF): a and b are half the weight, so that an infinity stays one and
// is not multiplied with 0.
template <int MODE, bool SELF>
__device__ __forceinline__ void coefficients(const float* weight, const float* row, int c0, bool live, int R,
                                             f32x2 (&ca)[4], f32x2 (&cb)[4]) {
  float w[8], a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.0f;
  if (weight != nullptr && live) load_f8(weight + c0, w);
  if (row != nullptr && c0 < R) {                  // R is a multiple of 16: a chunk is in or out
    float cs[8];
    if (adjacent(MODE)) {
      load_f8(row + c0, cs);
#pragma unroll
      for (int p = 0; p < 8; p += 2) {
        a[p] = w[p] * cs[p];
        b[p] = -w[p + 1] * cs[p + 1];
        a[p + 1] = w[p + 1] * cs[p];
        b[p + 1] = w[p] * cs[p + 1];
      }
    } else {
      const int half = R / 2;
      const bool upper = c0 >= half;
      const int other = upper ? c0 - half : c0 + half;
      const float sign = upper ? 1.0f : -1.0f;
      float wq[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) wq[j] = 1.0f;
      if (weight != nullptr) load_f8(weight + other, wq);
      row += 2 * (upper ? other : c0);
#pragma unroll
      for (int g = 0; g < 8; g += 4) {
        load_f8(row + 2 * g, cs);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          a[g + p] = w[g + p] * cs[2 * p];
          b[g + p] = sign * wq[g + p] * cs[2 * p + 1];
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = SELF ? 0.5f * w[j] : w[j];
      b[j] = SELF ? a[j] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ca[i] = pack_f32x2(a[pair_lo<MODE>(i)], a[pair_hi<MODE>(i)]);
    cb[i] = pack_f32x2(b[pair_lo<MODE>(i)], b[pair_hi<MODE>(i)]);
  }
}

template <int MODE, bool FP16>
__device__ __forceinline__ void unpack_chunk(const uint32_t (&w)[4], f32x2 (&f)[4]) {
  float e[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2<FP16>(w[i], e[2 * i], e[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pack_f32x2(e[pair_lo<MODE>(i)], e[pair_hi<MODE>(i)]);
}

template <int MODE, bool FP16>
__device__ __forceinline__ void pack_chunk(const f32x2 (&y)[4], uint32_t (&w)[4]) {
  float e[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_f32x2(y[i], e[pair_lo<MODE>(i)], e[pair_hi<MODE>(i)]);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<FP16>(e[2 * i], e[2 * i + 1]);
}

// A warp's work on one tensor: heads [h_first, h_end) of token t of batch row b, `heads` of them at a time; t and
// the lane's group among them (hsub) differ between groups that hold several tokens, alive = t is a token.
// Returns the largest |y| pattern (two 16-bit halves; only with a running amax) and sets bad for a non-finite value.
template <int G, int MODE, bool FP16, bool E4M3, bool PLAIN>
__device__ __forceinline__ uint32_t norm_rope_heads(const NormRopeArgs& args, const NormRopeSeg& sg, int b, int t,
                                                    bool alive, int hsub, int heads, int h_first, int h_end,
                                                    bool first, uint32_t ring, bool& bad) {
  const int lane = threadIdx.x & 31, gl = lane % G;
  const int second = (args.D / 8 + 1) / 2;         // chunk gl and chunk gl + second
  const int c0 = gl * 8, c1 = c0 + second * 8;
  const bool live0 = alive && gl < second, live1 = live0 && c1 < args.D;
  const bool norm = sg.weight != nullptr, track = !E4M3 && sg.amax != nullptr;

  const int64_t x_h = sg.x_h, o_h = sg.o_h;
  const uint16_t* x = static_cast<const uint16_t*>(sg.x) + b * sg.x_b + t * sg.x_t + (h_first + hsub) * x_h + c0;
  const int64_t x_step = heads * x_h;
  // step k of the warp's heads goes to slot k mod (depth + 1); the slot that a load overwrites was used one step ago
  int h_load = h_first;
  uint32_t slot_load = ring;
  const uint32_t ring_end = ring + (ROPE_DEPTH + 1) * ROPE_STEP_BYTES;
  auto load_step = [&] {
    if (h_load < h_end) {                          // uniform
      const bool in = h_load + hsub < h_end;
      cp_async16(slot_load, in && live0 ? x : static_cast<const uint16_t*>(sg.x), in && live0);
      cp_async16(slot_load + 512, in && live1 ? x + second * 8 : static_cast<const uint16_t*>(sg.x), in && live1);
      x += x_step;
      h_load += heads;
      slot_load = slot_load + ROPE_STEP_BYTES == ring_end ? ring : slot_load + ROPE_STEP_BYTES;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < ROPE_DEPTH; ++k) load_step();

  // E4M3: scale of the given amax (a non-finite amax writes no code).  Away from the ends of FP32 its
  // reciprocal goes into the norm's factor, behind the rotation: in the coefficients it could take products of large
  // values past FP32's range that cancel (PLAIN: into the correctly rounded quotient)
  float inv_s = 1.0f;
  CodeDiv cd{1.0f, true, 0, 0};
  if (E4M3) {
    const float amax = __ldg(sg.amax);
    if (!(fabsf(amax) <= 3.402823466e38f)) {              // inf or NaN
      cp_async_wait<0>();
      bad = true;
      return 0;
    }
    cd.s = amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f);
    const float r = __frcp_rn(cd.s);
    cd.rr = pack_f32x2(r, r);
    cd.ns = pack_f32x2(-cd.s, -cd.s);
    cd.fast = cd.s >= 0x1p-30f && cd.s <= 0x1p+30f;
    if (cd.fast) inv_s = r;
    if (first && lane == 0) *sg.scale_out = cd.s;
  }

  const int rotated = sg.table == nullptr ? 0 : args.R;      // ROT_PAIRS_PART
  f32x2 ca[2][4], cb[2][4];
  int src[2] = {lane, lane};                       // ROT_SHUFFLE: lane and chunk of the partners, itself without a rotation
  bool src1[2] = {false, true};
  if (!PLAIN) {
    const float* row = sg.table == nullptr ? nullptr : sg.table + b * sg.table_b + static_cast<int64_t>(t) * args.R;
    coefficients<MODE, MODE == ROT_LOW || MODE == ROT_SHUFFLE>(sg.weight, live0 ? row : nullptr, c0, live0, args.R, ca[0], cb[0]);
    coefficients<MODE, MODE == ROT_SHUFFLE>(sg.weight, live1 ? row : nullptr, c1, live1, args.R, ca[1], cb[1]);
    if (MODE == ROT_SHUFFLE || MODE == ROT_LOW) {
      const int half8 = args.R / 16;               // chunks of half the rotated channels
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int c = s == 0 ? gl : gl + second;
        if (row != nullptr && (s == 0 ? live0 : live1) && c < 2 * half8) {
          const int other = c < half8 ? c + half8 : c - half8;
          src1[s] = other >= second;
          src[s] = lane - gl + (src1[s] ? other - second : other);
        }
      }
    }
  }

  uint8_t* out = static_cast<uint8_t*>(sg.out) +
                 (b * sg.o_b + t * sg.o_t + (h_first + hsub) * o_h + c0) * (E4M3 ? 1 : 2);
  const int64_t o_step = heads * o_h * (E4M3 ? 1 : 2);
  uint32_t slot = ring;
  uint32_t m2 = 0, nan2 = 0;
  float bad32 = 0.0f;                              // + 0 * value: NaN once one is not finite
#pragma unroll 1
  for (int h0 = h_first; h0 < h_end; h0 += heads) {
    load_step();
    cp_async_wait<ROPE_DEPTH>();
    const bool in = h0 + hsub < h_end && QATTN_IN_BOUNDS(args.err, t < sg.L && h0 + hsub < sg.H);
    const uint4 v0 = ld_shared_v4(slot), v1 = ld_shared_v4(slot + 512);
    slot = slot + ROPE_STEP_BYTES == ring_end ? ring : slot + ROPE_STEP_BYTES;
    uint32_t w[2][4] = {{v0.x, v0.y, v0.z, v0.w}, {v1.x, v1.y, v1.z, v1.w}};
    uint32_t code[2][2];
    if (PLAIN) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan2 = note_nonfinite<FP16>(w[s][i], nan2);
      if (E4M3) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)            // the fast quotient of an infinity is NaN; the division saturates it
            code[s][i] = cd.fast && nan2 == 0 ? codes4<FP16, true>(w[s][2 * i], w[s][2 * i + 1], cd)
                                              : codes4<FP16, false>(w[s][2 * i], w[s][2 * i + 1], cd);
      }
    } else {
      f32x2 f[2][4], y[2][4];
      unpack_chunk<MODE, FP16>(w[0], f[0]);
      unpack_chunk<MODE, FP16>(w[1], f[1]);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (MODE == ROT_PAIRS_PART && (s == 0 ? c0 : c1) >= rotated) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[s][i] = mul_f32x2(ca[s][i], f[s][i]);
        } else if (adjacent(MODE)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[s][i] = fma_f32x2(cb[s][i], f[s][i ^ 2], mul_f32x2(ca[s][i], f[s][i]));
        } else if (MODE == ROT_HALVES) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[s][i] = fma_f32x2(cb[s][i], f[s ^ 1][i], mul_f32x2(ca[s][i], f[s][i]));
        } else if (MODE == ROT_LOW) {
          if (s == 0) {
            uint32_t q[4];
            f32x2 g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = __shfl_sync(0xFFFFFFFFu, w[0][i], src[0]);
            unpack_chunk<MODE, FP16>(q, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[0][i] = fma_f32x2(cb[0][i], g[i], mul_f32x2(ca[0][i], f[0][i]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[1][i] = mul_f32x2(ca[1][i], f[1][i]);
          }
        } else {
          uint32_t q[4];
          f32x2 g[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t q0 = __shfl_sync(0xFFFFFFFFu, w[0][i], src[s]), q1 = __shfl_sync(0xFFFFFFFFu, w[1][i], src[s]);
            q[i] = src1[s] ? q1 : q0;
          }
          unpack_chunk<MODE, FP16>(q, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[s][i] = fma_f32x2(cb[s][i], g[i], mul_f32x2(ca[s][i], f[s][i]));
        }
      }
      if (norm) {
        f32x2 s2 = mul_f32x2(f[0][0], f[0][0]), t2 = mul_f32x2(f[1][0], f[1][0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          s2 = fma_f32x2(f[0][i], f[0][i], s2);
          t2 = fma_f32x2(f[1][i], f[1][i], t2);
        }
        float ss, s1;
        unpack_f32x2(add_f32x2(s2, t2), ss, s1);
        ss += s1;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        bad32 = fmaf(ss, 0.0f, bad32);           // a non-finite element, or squares past FP32
        float r = rsqrtf(fmaf(ss, args.inv_d, args.eps));
        if (E4M3) r *= inv_s;
        const f32x2 r2 = pack_f32x2(r, r);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[s][i] = mul_f32x2(y[s][i], r2);
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            nan2 = note_nonfinite<FP16>(w[s][i], nan2);
            if (E4M3) y[s][i] = mul_f32x2(y[s][i], pack_f32x2(inv_s, inv_s));
          }
      }
      if (E4M3) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpack_f32x2(y[s][i], e[pair_lo<MODE>(i)], e[pair_hi<MODE>(i)]);
          if (!cd.fast) {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = __fdiv_rn(e[i], cd.s);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            code[s][i] = cvt_e4m3x2(e[4 * i], e[4 * i + 1]) | (cvt_e4m3x2(e[4 * i + 2], e[4 * i + 3]) << 16);
        }
      } else {
        pack_chunk<MODE, FP16>(y[0], w[0]);
        pack_chunk<MODE, FP16>(y[1], w[1]);
      }
    }
    if (E4M3) {
      if (in && live0) *reinterpret_cast<uint2*>(out) = make_uint2(code[0][0], code[0][1]);
      if (in && live1) *reinterpret_cast<uint2*>(out + second * 8) = make_uint2(code[1][0], code[1][1]);
    } else {
      if (in && live0) *reinterpret_cast<uint4*>(out) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
      if (in && live1) *reinterpret_cast<uint4*>(out + second * 16) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
      if (track) {                               // what is stored: a group without a head or token may hold 0 * inf
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (in && (s == 0 ? live0 : live1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, w[s][i] & 0x7FFF7FFFu);
          }
        }
      }
    }
    out += o_step;
  }
  bad |= nan2 != 0 || bad32 != 0.0f || bad32 != bad32;
  return m2;
}

template <int G, int MODE, bool FP16>
__global__ void __launch_bounds__(32 * ROPE_WARPS, ROPE_BLOCKS)
    k_norm_rope(const __grid_constant__ NormRopeArgs args) {
  extern __shared__ __align__(128) uint8_t rope_ring[];
  int si = 0;
  while (si + 1 < args.n && blockIdx.x >= args.seg[si + 1].first_block) ++si;
  const NormRopeSeg& sg = args.seg[si];
  const uint32_t item = (blockIdx.x - sg.first_block) * ROPE_WARPS + (threadIdx.x >> 5);
  uint32_t m2 = 0;
  bool bad = false;
  if (item < sg.items) {                           // warp-uniform
    // token fastest, so that the warps of a block write neighbouring rows of the same heads
    const uint32_t rest = item / sg.rows;
    const int b = static_cast<int>(rest / static_cast<uint32_t>(sg.chunks));
    const int group = (threadIdx.x & 31) / G, hsub = group & (sg.heads - 1);
    int t = static_cast<int>((item - rest * sg.rows) * sg.tokens) + (group >> sg.heads_log2);
    const bool alive = t < sg.L;
    if (!alive) t = 0;                             // its table row is not used either
    const int h_first = (static_cast<int>(rest) - b * sg.chunks) * sg.steps * sg.heads;
    const int h_end = min(sg.H, h_first + sg.steps * sg.heads);
    const bool plain = sg.weight == nullptr && sg.table == nullptr;
    const uint32_t ring = smem_u32(rope_ring) + (threadIdx.x >> 5) * ((ROPE_DEPTH + 1) * ROPE_STEP_BYTES) +
                          (threadIdx.x & 31) * 16;
    auto run = [&](auto e4m3, auto copy) {
      return norm_rope_heads<G, MODE, FP16, decltype(e4m3)::value, decltype(copy)::value>(
          args, sg, b, t, alive, hsub, sg.heads, h_first, h_end, item == 0, ring, bad);
    };
    using Yes = Flag<true>;
    using No = Flag<false>;
    if (sg.e4m3) m2 = plain ? run(Yes{}, Yes{}) : run(Yes{}, No{});
    else m2 = plain ? run(No{}, Yes{}) : run(No{}, No{});
  }
  const int lane = threadIdx.x & 31;
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicExch(args.err, DEV_ERR_NONFINITE);
  if (!sg.e4m3 && sg.amax != nullptr) {            // running amax: its order cannot change the result
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
    __shared__ uint32_t block_max;
    if (threadIdx.x == 0) block_max = 0;
    __syncthreads();
    if (lane == 0) atomicMax(&block_max, m);
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t mm = block_max;
      const float a = FP16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(mm)))
                           : __uint_as_float(mm << 16);
      if (mm >= (FP16 ? 0x7C00u : 0x7F80u)) atomicExch(args.err, DEV_ERR_NONFINITE);   // also by rounding
      // a >= 0, so that bit patterns compare as signed integers, with a negative start (-infinity) below all of them
      int* dst = reinterpret_cast<int*>(sg.amax);
      if (__float_as_int(a) > *static_cast<volatile int*>(dst)) atomicMax(dst, __float_as_int(a));
    }
  }
}

// Lanes of a head's group: two chunks of eight channels each.
static int group_lanes(int D) { return D <= 64 ? 4 : D <= 128 ? 8 : 16; }

static_assert(ROPE_SMEM <= 48 * 1024, "no attribute is set for more");

template <int G, int MODE>
static cudaError_t launch_g(const NormRopeArgs& a, unsigned grid, bool fp16, cudaStream_t stream) {
  if (fp16) k_norm_rope<G, MODE, true><<<grid, 32 * ROPE_WARPS, ROPE_SMEM, stream>>>(a);
  else k_norm_rope<G, MODE, false><<<grid, 32 * ROPE_WARPS, ROPE_SMEM, stream>>>(a);
  return cudaGetLastError();
}

// A warp has 32 / G groups of lanes, for `heads` heads (a power of two) of each of `tokens` tokens, and takes `steps`
// such steps.  Forming a token's coefficients costs a group about as much as a step, so one head of several tokens at
// a time and many steps are best (8704 x 24 heads as E4M3 48.9 -> 43.6 us, 12624 x 16 and 4 heads of 64 25.0 -> 16.9); with fewer tokens, fewer steps and then
// more heads at a time keep 64 warps for every SM, down to one step of all groups' heads for a single token.
bool plan_norm_rope(NormRopeArgs& a, int B, int num_sms, unsigned* grid) {
  const int groups = 32 / group_lanes(a.D);
  const int64_t want = static_cast<int64_t>(num_sms) * 64;      // warps
  int heads = 1, most = 16;
  int64_t blocks = 0;
  for (;;) {
    int64_t items = 0;
    blocks = 0;
    for (int i = 0; i < a.n; ++i) {
      NormRopeSeg& s = a.seg[i];
      s.heads_log2 = 0;
      while ((1 << s.heads_log2) < s.H && (1 << s.heads_log2) < heads) ++s.heads_log2;
      s.heads = 1 << s.heads_log2;
      s.tokens = groups / s.heads;
      s.rows = static_cast<uint32_t>((s.L - 1) / s.tokens + 1);
      const int all = (s.H - 1) / s.heads + 1;
      s.chunks = (all - 1) / most + 1;
      s.steps = (all - 1) / s.chunks + 1;
      const int64_t mine = static_cast<int64_t>(B) * s.rows * s.chunks;
      if (mine > 0xFFFFFFF0ll - ROPE_WARPS) return false;
      s.items = static_cast<uint32_t>(mine);
      s.first_block = static_cast<unsigned>(blocks);
      items += mine;
      blocks += (mine + ROPE_WARPS - 1) / ROPE_WARPS;
      if (blocks > 0x7FFFFFFF) return false;
    }
    if (items >= want || (heads == groups && most == 1)) break;
    if (most > 4 || heads == groups) most /= 2;
    else heads *= 2;
  }
  *grid = static_cast<unsigned>(blocks);
  return true;
}

template <int MODE>
static cudaError_t launch_mode(const NormRopeArgs& a, unsigned grid, bool fp16, cudaStream_t stream) {
  switch (group_lanes(a.D)) {
    case 4: return launch_g<4, MODE>(a, grid, fp16, stream);
    case 8: return launch_g<8, MODE>(a, grid, fp16, stream);
    default: return launch_g<16, MODE>(a, grid, fp16, stream);
  }
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, unsigned grid, int pairs, int fp16, cudaStream_t stream) {
  bool whole = a.R == a.D;                         // every channel that is computed is rotated
  for (int i = 0; i < a.n; ++i) whole = whole && (a.seg[i].weight == nullptr || a.seg[i].table != nullptr);
  if (pairs && whole) return launch_mode<ROT_PAIRS>(a, grid, fp16 != 0, stream);
  if (pairs && a.R > 0) return launch_mode<ROT_PAIRS_PART>(a, grid, fp16 != 0, stream);   // R = 0: ROT_LOW, 1 % faster
  // a whole head rotated by halves: its partner chunks are D / 16 apart, as a lane's two chunks are
  if (whole) return launch_mode<ROT_HALVES>(a, grid, fp16 != 0, stream);
  if (a.R / 8 <= (a.D / 8 + 1) / 2) return launch_mode<ROT_LOW>(a, grid, fp16 != 0, stream);
  return launch_mode<ROT_SHUFFLE>(a, grid, fp16 != 0, stream);
}

}  // namespace qattn
