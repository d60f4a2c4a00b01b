// Products of stored weight rows with a few token rows on the matrix cores:
// the part that fp4_matvec and moe_layer_few share.
//
// acc[f][n] (16 weight rows x 16 tokens, fp32) += W_f[16, K] x_n[16, K]^T for
// RT row tiles and NT token tiles.  With few tokens the work is reading W
// once, so the kernel is a stream: weights go from memory to registers with
// 16-byte loads and never pass through LDS, each step's loads are issued D
// steps ahead, and the waves of a block share the K axis, which keeps many
// bytes in flight; their sums meet in LDS at the end.
//
// K order.  A step is LD loads of 16 bytes per lane.  Lane l works on weight
// row l % 16 and on 16-byte chunk c = (step LD + load) 4 + l / 16 of it, i.e.
// on K indices [c EPL, (c + 1) EPL); its token column l % 16 reads the same
// indices of x.  Any order of K inside a matrix instruction then pairs equal
// indices.  A chunk that starts at or past K is not fetched and counts as
// zeros on both sides, as do rows and tokens that do not exist, so nothing is
// read out of bounds and a NaN in one row or token stays in its own results.
//
// Few tokens of a narrow type.  A chunk of E4M3 or E2M1 weights meets 32 or 64
// bytes of x, XV loads of 16 bytes a lane, of which one token fills only the
// lanes of one column: x then costs more load instructions than the weights.
// Packed (PK), up to 16 / XV tokens share one load: column t XV + v holds
// piece v of token t, the products of the weights' piece v go to accumulator
// v, and the sum of a token is that of its XV columns, column t XV + v taken
// from accumulator v.  What the other columns of an accumulator hold is not
// used.
//
// Weight types: fp32 (fp32 matrix instructions); bf16; E4M3 with one scale
// per 128x128 block; E2M1 with one exponent byte per 32 columns of a row,
// exactly one lane's chunk.  The two narrow types are widened to bf16 by the
// scaled conversions, which apply the power-of-two scale exactly.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 sk_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 sk_bf16x2 __attribute__((ext_vector_type(2)));
typedef float sk_f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned sk_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned sk_u32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t SK_OOB = 0x80000000u;  // past the end of any buffer below 2 GiB

__device__ __forceinline__ __amdgpu_buffer_rsrc_t sk_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

template <int WT>
struct SkinnyWeight;
template <>
struct SkinnyWeight<MOE_F32> {
  static constexpr int EPL = 4, LD = 2;
};
template <>
struct SkinnyWeight<MOE_BF16> {
  static constexpr int EPL = 8, LD = 2;
};
template <>
struct SkinnyWeight<MOE_E4M3> {
  static constexpr int EPL = 16, LD = 2;  // a step is one 128-wide scale block
};
template <>
struct SkinnyWeight<MOE_E2M1> {
  static constexpr int EPL = 32, LD = 1;
};

// Bytes of a row of K weights of type WT.
__host__ __device__ constexpr long long sk_row_bytes(int wt, long long K) {
  return wt == MOE_F32 ? K * 4 : wt == MOE_BF16 ? K * 2 : wt == MOE_E4M3 ? K : K / 2;
}

__device__ __forceinline__ sk_bf16x8 sk_join(sk_bf16x2 a, sk_bf16x2 b, sk_bf16x2 c, sk_bf16x2 d) {
  return sk_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// SV: the exponent bytes of E2M1 weights are read 16 at a time, four steps'
// worth of a row's, which needs rows of a multiple of 4 bytes (K % 128 == 0);
// otherwise a byte a step.
template <int WT, typename XT, int RT, int NT, bool SV = false, bool PK = false>
struct Skinny {
  static_assert(!SV || WT == MOE_E2M1, "only E2M1 has exponent bytes");
  static constexpr int EPL = SkinnyWeight<WT>::EPL, LD = SkinnyWeight<WT>::LD;
  static constexpr int STEP = 4 * EPL * LD;                             // K indices per step
  static constexpr int XBYTES = EPL * (int)sizeof(XT);                  // x bytes of a chunk: 8, 16, 32 or 64
  static constexpr int XV = XBYTES < 16 ? 1 : XBYTES / 16;              // 16-byte pieces of it
  static constexpr int XL = PK ? 1 : XV;                                // loads of it
  static constexpr int AC = PK ? XV : NT;                               // accumulators of a row tile
  static constexpr int TOKENS = PK ? 16 / XV : 16 * NT;                 // tokens at a time
  static_assert(!PK || NT == 1, "one tile of columns");
  static_assert(WT == MOE_F32 || sizeof(XT) == 2, "narrow weights take bf16 tokens");

  // Whether a tile of tokens j0 .. j0 + TOKENS - 1 of `toks` holds the sums of
  // column lane % 16: a packed tile holds fewer tokens than it has columns, and
  // what sk_get_packed finds for the others is another row group's or no one's.
  __host__ __device__ static constexpr bool holds(int lane, int j0, int toks) {
    return (lane & 15) < TOKENS && j0 + (lane & 15) < toks;
  }

  struct Lanes {
    __amdgpu_buffer_rsrc_t rw, rs, rx;
    uint32_t w_off[RT];  // byte offset of the lane's row of tile f, chunk l / 16 included; SK_OOB: no such row
    uint32_t s_off[RT];  // E2M1: byte offset of its exponent bytes (SV: the row's, else chunk l / 16 included)
    uint32_t x_off[NT];  // byte offset of the lane's token row, chunk l / 16 (PK: and piece) included; SK_OOB: none
    const float* blk_lo;  // E4M3: scales along K of the 128-row block of tiles f < RT / 2, and of the others
    const float* blk_hi;
    int K, g;
  };
  struct Step {
    sk_u32x4 w[RT][LD];
    sk_u32x4 x[NT][LD][XL];
    uint32_t s[RT];
    float blk[2];
  };
  struct Scales {
    sk_u32x4 v[RT];  // word i: the exponent bytes of step i of four
  };

  __device__ static __forceinline__ void load_scales(Scales& sc, const Lanes& L, int s) {
#pragma unroll
    for (int f = 0; f < RT; ++f) sc.v[f] = __builtin_amdgcn_raw_buffer_load_b128(L.rs, L.s_off[f], (uint32_t)s * 4u, 0);
  }

  __device__ static __forceinline__ uint32_t past_k(const Lanes& L, uint32_t c) {
    return (int)(c + L.g) * EPL < L.K ? 0u : SK_OOB;
  }
  // First chunk of load l of step s as a scalar offset, which has to stay
  // within the buffer: 0 where the whole load lies past K (its lanes are past
  // the end by their own offsets).
  __device__ static __forceinline__ uint32_t base_chunk(const Lanes& L, uint32_t c) {
    return (int)c * EPL < L.K ? c : 0u;
  }

  __device__ static __forceinline__ void load_w(Step& st, const Lanes& L, int s) {
#pragma unroll
    for (int l = 0; l < LD; ++l) {
      const uint32_t first = (uint32_t)(s * LD + l) * 4u, c = base_chunk(L, first);
      const uint32_t oob = past_k(L, first);
#pragma unroll
      for (int f = 0; f < RT; ++f)
        st.w[f][l] = __builtin_amdgcn_raw_buffer_load_b128(L.rw, L.w_off[f] | oob, c * 16u, 0);
      if (WT == MOE_E2M1 && !SV) {
#pragma unroll
        for (int f = 0; f < RT; ++f) st.s[f] = __builtin_amdgcn_raw_buffer_load_b8(L.rs, L.s_off[f] | oob, c, 0);
      }
    }
    if (WT == MOE_E4M3) {
      const int b = s < (L.K >> 7) ? s : 0;
      st.blk[0] = L.blk_lo[b];
      st.blk[1] = L.blk_hi[b];
    }
  }

  __device__ static __forceinline__ void load_x(sk_u32x4 (&x)[NT][LD][XL], const Lanes& L, int s) {
#pragma unroll
    for (int l = 0; l < LD; ++l) {
      const uint32_t first = (uint32_t)(s * LD + l) * 4u, c = base_chunk(L, first);
      const uint32_t oob = past_k(L, first);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t xo = L.x_off[n] | oob;
        if (XBYTES < 16) {
          const sk_u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(L.rx, xo, c * XBYTES, 0);
          x[n][l][0] = sk_u32x4{v[0], v[1], 0u, 0u};
        } else {
#pragma unroll
          for (int v = 0; v < XL; ++v)
            x[n][l][v] = __builtin_amdgcn_raw_buffer_load_b128(L.rx, xo, c * XBYTES + v * 16u, 0);
        }
      }
    }
  }

  __device__ static __forceinline__ void load(Step& st, const Lanes& L, int s) {
    load_w(st, L, s);
    load_x(st.x, L, s);
  }

  __device__ static __forceinline__ void mma(sk_f32x4 (&acc)[RT][AC], const Step& st, const Lanes& L, const Scales& sv,
                                             int i4) {
#pragma unroll
    for (int l = 0; l < LD; ++l) {
      if constexpr (WT == MOE_F32) {
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[n][i] = sizeof(XT) == 4 ? __uint_as_float(st.x[n][l][0][i])
                      : (i & 1)       ? __uint_as_float(st.x[n][l][0][i >> 1] & 0xFFFF0000u)
                                      : __uint_as_float(st.x[n][l][0][i >> 1] << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int f = 0; f < RT; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(st.w[f][l][i]), x[n][i], acc[f][n], 0, 0, 0);
      } else {
#pragma unroll
        for (int f = 0; f < RT; ++f) {
          sk_bf16x8 a[EPL / 8];
          if constexpr (WT == MOE_BF16) {
            a[0] = __builtin_bit_cast(sk_bf16x8, st.w[f][l]);
          } else if constexpr (WT == MOE_E4M3) {
            const float sc = st.blk[f < RT / 2 ? 0 : 1];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              a[j] = sk_join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(st.w[f][l][2 * j], sc, false),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(st.w[f][l][2 * j], sc, true),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(st.w[f][l][2 * j + 1], sc, false),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(st.w[f][l][2 * j + 1], sc, true));
          } else {
            const uint32_t b = SV ? (sv.v[f][i4] >> (8 * L.g)) & 0xFFu : st.s[f];
            const float sc = __uint_as_float(b << 23);  // E8M0: 2^(byte - 127)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[j] = sk_join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(st.w[f][l][j], sc, 0),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(st.w[f][l][j], sc, 1),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(st.w[f][l][j], sc, 2),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(st.w[f][l][j], sc, 3));
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < EPL / 8; ++j) {
              sk_f32x4& c = acc[f][PK ? j % XV : n];
              c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], __builtin_bit_cast(sk_bf16x8, st.x[n][l][PK ? 0 : j]), c,
                                                          0, 0, 0);
            }
        }
      }
    }
  }

  // Steps s0 to s1 - 1, loads D steps ahead, those of G steps together.  The
  // branches are uniform: no step past the end is loaded or multiplied (a wave
  // has few steps, so rounding their number up to D costs more than the
  // branches).
  template <int D, int G = 1>
  __device__ static __forceinline__ void run(sk_f32x4 (&acc)[RT][AC], const Lanes& L, int s0, int s1) {
    constexpr int U = SV ? 4 : D;  // steps to a turn of the loop: a vector holds the exponent bytes of four
    static_assert(U % D == 0 && D % G == 0, "a turn of the loop goes round the ring");
#pragma unroll
    for (int f = 0; f < RT; ++f)
#pragma unroll
      for (int n = 0; n < AC; ++n) acc[f][n] = sk_f32x4{0.f, 0.f, 0.f, 0.f};
    s0 = __builtin_amdgcn_readfirstlane(s0);
    s1 = __builtin_amdgcn_readfirstlane(s1);
    Step st[D];
    Scales sc[2];
    if (SV) load_scales(sc[0], L, s0);
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (s0 + i < s1) load(st[i], L, s0 + i);
      __builtin_amdgcn_sched_barrier(0);
    }
    int s = s0;
    for (; s + U + D - 1 < s1; s += U) {
      if (SV) load_scales(sc[1], L, s + U);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        mma(acc, st[i % D], L, sc[0], i);
        __builtin_amdgcn_sched_barrier(0);
        if (i % G == G - 1)
#pragma unroll
          for (int j = i - G + 1; j <= i; ++j) load(st[j % D], L, s + D + j);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (SV) sc[0] = sc[1];
    }
    if (SV && s + U < s1) load_scales(sc[1], L, s + U);
#pragma unroll
    for (int i = 0; i < U + D - 1; ++i) {
      if (s + i < s1) mma(acc, st[i % D], L, sc[i / U], i % U);
      __builtin_amdgcn_sched_barrier(0);
      if (i < U && i % G == G - 1)
#pragma unroll
        for (int j = i - G + 1; j <= i; ++j)
          if (s + D + j < s1) load(st[j % D], L, s + D + j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Wave w of W: steps [s0, s1) cut into W runs of equal length (or one less).
  template <int D, int G = 1>
  __device__ static __forceinline__ void run_part(sk_f32x4 (&acc)[RT][AC], const Lanes& L, int s0, int s1, int w, int W) {
    const int n = s1 > s0 ? s1 - s0 : 0;
    run<D, G>(acc, L, s0 + n * w / W, s0 + n * (w + 1) / W);
  }
};

// The W waves' accumulators of one block, added in the order of the waves.
// Element (f, n, lane) of the sum: rows 4 (lane / 16) + 0..3 of tile f, token
// lane % 16 of tile n.
template <int RT, int NT>
__device__ __forceinline__ void sk_put(sk_f32x4* red, const sk_f32x4 (&acc)[RT][NT], int tid) {
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[((wave * RT + f) * NT + n) * 64 + lane] = acc[f][n];
  __syncthreads();
}
template <int W, int RT, int NT>
__device__ __forceinline__ sk_f32x4 sk_get(const sk_f32x4* red, int f, int n, int lane) {
  sk_f32x4 s = red[(f * NT + n) * 64 + lane];
#pragma unroll
  for (int w = 1; w < W; ++w) s += red[((w * RT + f) * NT + n) * 64 + lane];
  return s;
}

// The same for packed tokens (token lane % 16, below 16 / XV): one tile of
// columns a wave, each from its own accumulator.
template <int RT, int XV>
__device__ __forceinline__ void sk_put_packed(sk_f32x4* red, const sk_f32x4 (&acc)[RT][XV], int tid) {
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int f = 0; f < RT; ++f) {
    sk_f32x4 v = acc[f][0];
#pragma unroll
    for (int n = 1; n < XV; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lane % XV == n ? acc[f][n][i] : v[i];
    red[(wave * RT + f) * 64 + lane] = v;
  }
  __syncthreads();
}
// Its first column of the 64 values of a wave's row tile.
template <int XV>
__host__ __device__ constexpr int sk_packed_at(int lane) {
  return (lane & 48) + (lane & 15) * XV;
}
template <int W, int RT, int XV>
__device__ __forceinline__ sk_f32x4 sk_get_packed(const sk_f32x4* red, int f, int lane) {
  const int at = sk_packed_at<XV>(lane);
  sk_f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < W; ++w) {
    sk_f32x4 v = red[(w * RT + f) * 64 + at];
#pragma unroll
    for (int n = 1; n < XV; ++n) v += red[(w * RT + f) * 64 + at + n];
    s = w ? s + v : v;
  }
  return s;
}

}  // namespace moe
