// The adapters' second product and the output of q8ta_linear_lora, for the
// 32x32x32 matrix-core GEMMs: what a wave does with its integer sums instead of
// requantizing them.
#pragma once

#include <type_traits>

#include "decode.h"

namespace q8ta {

struct NoLora {
  static constexpr bool kOn = false;
};
template <class AT_, class YT_>
struct WithLora {
  static constexpr bool kOn = true;
  typedef AT_ AT;
  typedef YT_ YT;
  LoraArgs l;
};
// launch<EP>() for the adapter and output types of a.
template <class F>
inline hipError_t lora_types(const LoraArgs& a, F&& launch) {
  if (a.ad_type == Q8TA_F16) {
    if (a.y_type == Q8TA_F32) return launch(WithLora<Half, float>{a});
    if (a.y_type == Q8TA_F16) return launch(WithLora<Half, Half>{a});
    return launch(WithLora<Half, Bfloat>{a});
  }
  if (a.y_type == Q8TA_F32) return launch(WithLora<Bfloat, float>{a});
  if (a.y_type == Q8TA_F16) return launch(WithLora<Bfloat, Half>{a});
  return launch(WithLora<Bfloat, Bfloat>{a});
}

typedef __bf16 lora_v8b __attribute__((ext_vector_type(8)));
typedef float lora_v16f __attribute__((ext_vector_type(16)));
typedef int lora_v16i __attribute__((ext_vector_type(16)));
typedef uint32_t lora_v4u __attribute__((ext_vector_type(4)));

// Eight values of B's row from rank r on, zero from the adapter's own rank on.
template <class AT>
__device__ __forceinline__ lora_v4u lora_b8(const AT* b, int r, int rank, bool vec) {
  lora_v4u w = lora_v4u{0, 0, 0, 0};
  if (vec) {
    if (r < rank) w = *reinterpret_cast<const lora_v4u*>(b + r);
    if (r < rank && r + 8 > rank) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] &= (r + 2 * e < rank ? 0xffffu : 0u) | (r + 2 * e + 1 < rank ? 0xffff0000u : 0u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (r + e < rank) w[e / 2] |= (uint32_t)b[r + e].bits << (16 * (e % 2));
  }
  return w;
}

// Non-zero where a value of the eight is infinite or NaN: an exponent of ones
// carries into the sign's place.
template <class AT>
__device__ __forceinline__ uint32_t not_finite(const lora_v4u& w) {
  constexpr uint32_t e = std::is_same<AT, Half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t one = std::is_same<AT, Half>::value ? 0x04000400u : 0x00800080u;
  uint32_t carry = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) carry |= (w[i] & e) + one;
  return carry & 0x80008000u;
}

// y += t B^T for the 64 rows and 32 * FN channels of a wave's fragments.  The
// rows' adapters are taken one after the other; rows of another adapter have a
// t of zero.  t comes as three bf16 parts, which hold all of its 24 bits (two hold
// 17: 2048 x 4096 x 11008 with rank 64 3 us less of 151, but outputs whose rank
// terms cancel are off by up to 70 times what 32 bits leave), B goes on as one part where it is bf16
// and as two, which hold all of its 11 bits, where it is fp16: bf16 has fp32's
// range, so t needs no scaling.  Products of parts below 2^-24 of the whole are
// left out.  Operands come straight from memory (16 bytes a lane).
template <class AT, int FN>
__device__ __forceinline__ void lora_add(const LoraArgs& l, lora_v16f (&y)[FN][2], int64_t row0,
                                         int64_t ch0, int lane) {
  constexpr int Q = std::is_same<AT, Half>::value ? 2 : 1;
  constexpr int P = kLoraParts;
  const int lrow = lane & 31, kg = lane >> 5;
  const int64_t N = l.lin.N, plane = l.lin.M * l.rank_pad;
  const bool vec = l.rank % 8 == 0 && ((uintptr_t)l.b & 15) == 0;
  const int id = row0 + lane < l.lin.M ? adapter_of(l, row0 + lane) : -1;
  const lora_v4u zero = lora_v4u{0, 0, 0, 0};
  uint64_t left = __ballot(id >= 0);
  while (left != 0) {
    const int ad = __builtin_amdgcn_readlane(id, (uint32_t)__builtin_ctzll(left));
    const uint64_t mine = __ballot(id == ad);
    left &= ~mine;
    const int rank = rank_of(l, ad);
    const AT* bb = (const AT*)l.b + (int64_t)ad * N * l.rank;
    const uint16_t* t = l.tp + (row0 + lrow) * l.rank_pad + 8 * kg;
    const bool in0 = (mine >> lrow) & 1, in1 = (mine >> (32 + lrow)) & 1;
    uint32_t odd = 0;   // bit i: this lane's channel of fragment i has such a value
    for (int r0 = 0; r0 < rank; r0 += 16) {
      lora_v4u tf[2][P], w[FN];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        tf[0][p] = zero;
        tf[1][p] = zero;
        if (in0) tf[0][p] = *reinterpret_cast<const lora_v4u*>(t + p * plane + r0);
        if (in1) tf[1][p] = *reinterpret_cast<const lora_v4u*>(t + p * plane + 32 * l.rank_pad + r0);
      }
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int64_t n = ch0 + 32 * i + lrow < N ? ch0 + 32 * i + lrow : N - 1;
        w[i] = lora_b8<AT>(bb + n * l.rank, r0 + 8 * kg, rank, vec);
      }
      // a value that is not finite would spoil the tile's rows of other
      // adapters (0 * inf): left out here, and its own rows become NaN below
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const uint32_t bad = not_finite<AT>(w[i]);
        if (__any(bad != 0)) {
          if (bad) w[i] = zero;
          odd |= bad ? 1u << i : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        lora_v4u bf[Q];
        if constexpr (Q == 1) {
          bf[0] = w[i];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t pair = w[i][e];
            const float lo = to_float(Half{(uint16_t)pair});
            const float hi = to_float(Half{(uint16_t)(pair >> 16)});
            const Bfloat l0 = from_float<Bfloat>(lo), h0 = from_float<Bfloat>(hi);
            const Bfloat l1 = from_float<Bfloat>(lo - to_float(l0));
            const Bfloat h1 = from_float<Bfloat>(hi - to_float(h0));
            bf[0][e] = (uint32_t)l0.bits | (uint32_t)h0.bits << 16;
            bf[1][e] = (uint32_t)l1.bits | (uint32_t)h1.bits << 16;
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int q = 0; q < Q && p + q < P; ++q) {
              const lora_v4u tv = tf[j][p], bv = bf[q];
              y[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  __builtin_bit_cast(lora_v8b, tv), __builtin_bit_cast(lora_v8b, bv), y[i][j], 0, 0, 0);
            }
      }
    }
    if (__any(odd != 0)) {
      odd |= __shfl_xor(odd, 32);
      const uint32_t own[2] = {(uint32_t)mine >> (4 * kg), (uint32_t)(mine >> 32) >> (4 * kg)};
      // a NaN's bits where the bit is set
      auto nan_if = [](uint32_t bits, int at) { return (bits >> at & 1) * 0x7fc00000u; };
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float v = y[i][j][r];   // (a bit cast of a vector's element reads element 0)
            const uint32_t nan = nan_if(odd, i) & nan_if(own[j], 8 * (r / 4) + r % 4);
            y[i][j][r] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) | nan);
          }
    }
  }
}

// Rounds and stores a wave's fragments, row by row of the registers.
template <class YT, int FN>
__device__ __forceinline__ void lora_put(const LoraArgs& l, const lora_v16f (&y)[FN][2],
                                         int64_t row0, int64_t ch0, int lane) {
  const int lrow = lane & 31, kg = lane >> 5;
  const int64_t M = l.lin.M, N = l.lin.N;
  const float low = l.relu ? 0.0f : -__builtin_inff();
  YT* out = (YT*)l.y;
  if (row0 + 64 <= M && ch0 + 32 * FN <= N && M * N <= (int64_t)INT32_MAX) {
    // interior: one 32-bit offset a lane, wave-uniform row bases
    const uint32_t off = (uint32_t)((row0 + 4 * kg) * N + ch0 + lrow);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        YT* rb = out + (int64_t)(32 * j + 8 * (r / 4) + r % 4) * N;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const float v = y[i][j][r];
          rb[off + 32 * i] = from_float<YT>(v < low ? low : v);
        }
      }
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t m = row0 + 32 * j + 8 * (r / 4) + 4 * kg + r % 4;
      YT* rb = out + m * N + ch0 + lrow;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const float v = y[i][j][r];
        if (m < M && ch0 + 32 * i + lrow < N) rb[32 * i] = from_float<YT>(v < low ? low : v);
      }
    }
}

// A wave's 64 rows from row0 and 32 * FN channels from ch0: register r of
// fragment (i, j) is row 32j + 8(r / 4) + 4(lane / 32) + r % 4 and channel 32i +
// lane % 32; zc, sc, bi: the channels' zero-point term, scale and bias.
template <class AT, class YT, int FN>
__device__ __forceinline__ void lora_finish(const LoraArgs& l, const lora_v16i (&acc)[FN][2],
                                            const int32_t (&zc)[FN], const float (&sc)[FN],
                                            const float (&bi)[FN], int64_t row0, int64_t ch0,
                                            int lane) {
  lora_v16f y[FN][2];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float v = (float)(acc[i][j][r] - zc[i]);
        v = v * l.lin.rq.s_in;
        v = v * sc[i];
        y[i][j][r] = v + bi[i];
      }
  lora_add<AT>(l, y, row0, ch0, lane);
  lora_put<YT>(l, y, row0, ch0, lane);
}

}  // namespace q8ta
