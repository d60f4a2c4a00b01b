// 4-bit weights: E2M1 codes with one power-of-two scale per 32 columns of a
// row (the group size and the element and scale formats of the OCP
// Microscaling specification's 4-bit format), their quantiser, and products
// with a few token rows.
#include "skinny.h"
#include "vec8.h"

namespace moe {

namespace {

// Smallest 2^k (k >= -126) with amax <= 6 * 2^k, or k = 0 for amax == 0: with
// amax = 1.M * 2^E, k = E - 2 when 1.M <= 1.5, else E - 1.  b: bits of amax.
__device__ __forceinline__ int e2m1_scale_exp(uint32_t b) {
  if (b == 0) return 0;
  const int E = (int)(b >> 23) - 127;
  if (E == -127) return -126;  // subnormal amax
  const int k = (b & 0x7FFFFFu) <= 0x400000u ? E - 2 : E - 1;
  return k < -126 ? -126 : k;
}

// Blocks of a launch: fewer than 2^32 threads, further chunks in a loop.
unsigned chunk_blocks(long long chunks) {
  const long long need = ceil_div(chunks, 256), most = 0xFFFFFFFFLL / 256;
  return (unsigned)(need < most ? need : most);
}

// Eight values per thread; four threads hold a group of 32.  The scaled
// conversion divides by the power of two exactly and rounds to nearest, a tie
// to the even code.  Bound by HBM: 65536 x 7168 fp32 values 367 us (5.8 TB/s),
// bf16 215 us (5.5 TB/s); with the codes from seven comparisons a value 429 and
// 360.
template <typename XT>
__global__ __launch_bounds__(256) void k_fp4_quant(const XT* __restrict__ x, long long chunks, uint8_t* __restrict__ q,
                                                   uint8_t* __restrict__ scale) {
  // chunks % 4 == 0: a group is live or not as one
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (long long)gridDim.x * 256) {
    float v[8];
    Vec8<XT>::load(x + i * 8, v);
    // the largest magnitude as an integer: infinities and NaN come out on top
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, 64));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, 64));
    const bool finite = amax < 0x7F800000u;
    const int k = finite ? e2m1_scale_exp(amax) : 0;
    const float sc = exp2_int(k);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
    *reinterpret_cast<uint32_t*>(q + i * 4) = finite ? w : 0u;
    if ((i & 3) == 0) scale[i >> 2] = finite ? (uint8_t)(k + 127) : 255;
  }
}

// Bound by HBM: 65536 x 7168 values to bf16 213 us (5.6 TB/s), to fp32 390.
template <typename OT>
__global__ __launch_bounds__(256) void k_fp4_dequant(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                     long long chunks, OT* __restrict__ out) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (long long)gridDim.x * 256) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q + i * 4);
    const float sc = __uint_as_float((uint32_t)scale[i >> 2] << 23);
    float v[8];
    auto put = [&](sk_bf16x2 p, int j) {  // exact: one significant bit beside the leading one
      v[j] = static_cast<float>(p[0]);
      v[j + 1] = static_cast<float>(p[1]);
    };
    put(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0), 0);
    put(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1), 2);
    put(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2), 4);
    put(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3), 6);
    Vec8<OT>::store(out + i * 8, v);
  }
}

template <typename OT>
__device__ __forceinline__ void mv_store(OT* o, const sk_f32x4& s, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) {
      if constexpr (sizeof(OT) == 2)
        o[i] = f32_to_bf16(s[i]);
      else
        o[i] = s[i];
    }
}

// One block: RT 16-row tiles of W and up to 16 NT tokens (PK: 4), its waves
// sharing the K axis.  4096 x 7168 and one token 5.9 us, 2.6 TB/s: launch and
// one latency of the stream bound it; 16384 x 7168 16 us, 3.9 TB/s (13 where
// the 256 MB last-level cache still holds the weights).  More than 4 tokens are
// bound by x, of which every wave reads its part from L2 for itself, 4 (16
// tokens) or 8 bytes (32) for a byte of a row tile's weights: 4096 rows 12 and
// 18 us, 16384 rows 22 and 29.
constexpr int MV_W = 8;  // waves

template <int RT, int NT, bool SV, bool PK, typename OT>
__global__ __launch_bounds__(64 * MV_W) void k_fp4_matvec(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, int T, long long N, int K,
                                                          OT* __restrict__ y) {
  using S = Skinny<MOE_E2M1, uint16_t, RT, NT, SV, PK>;
  __shared__ sk_f32x4 red[MV_W * RT * NT * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long row0 = (long long)blockIdx.x * (16 * RT);
  const int rows = (int)(N - row0 < 16 * RT ? N - row0 : 16 * RT);
  const int t0 = blockIdx.y * S::TOKENS;
  const int toks = T - t0 < S::TOKENS ? T - t0 : S::TOKENS;
  typename S::Lanes L;
  L.K = K;
  L.g = lane >> 4;
  L.rw = sk_rsrc(q + row0 * (K / 2), (uint32_t)rows * (uint32_t)(K / 2));
  L.rs = sk_rsrc(scale + row0 * (K / 32), (uint32_t)rows * (uint32_t)(K / 32));
  L.rx = sk_rsrc(x + (long long)t0 * K, (uint32_t)toks * (uint32_t)K * 2u);
#pragma unroll
  for (int f = 0; f < RT; ++f) {
    const int r = f * 16 + (lane & 15);
    L.w_off[f] = r < rows ? (uint32_t)r * (uint32_t)(K / 2) + L.g * 16u : SK_OOB;
    L.s_off[f] = r < rows ? (uint32_t)r * (uint32_t)(K / 32) + (SV ? 0 : L.g) : SK_OOB;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = PK ? (lane & 15) / S::XV : n * 16 + (lane & 15);
    L.x_off[n] = t < toks ? (uint32_t)t * (uint32_t)K * 2u + L.g * (uint32_t)S::XBYTES +
                                (PK ? (uint32_t)(lane % S::XV) * 16u : 0u)
                          : SK_OOB;
  }
  sk_f32x4 acc[RT][S::AC];
  S::template run_part<2>(acc, L, 0, (K + S::STEP - 1) / S::STEP, wave, MV_W);
  if constexpr (PK)
    sk_put_packed<RT, S::XV>(red, acc, threadIdx.x);
  else
    sk_put<RT, NT>(red, acc, threadIdx.x);
  for (int e = threadIdx.x; e < RT * NT * 64; e += 64 * MV_W) {
    const int l = e & 63, n = (e >> 6) % NT, f = (e >> 6) / NT;
    const int t = n * 16 + (l & 15), r = f * 16 + 4 * (l >> 4);
    if (t >= toks || r >= rows) continue;
    sk_f32x4 s;
    if constexpr (PK)
      s = sk_get_packed<MV_W, RT, S::XV>(red, f, l);
    else
      s = sk_get<MV_W, RT, NT>(red, f, n, l);
    mv_store(y + (long long)(t0 + t) * N + row0 + r, s, rows - r);
  }
}

// Many rows and several tokens: the waves of a block take 16 RT rows each over
// the whole K axis and share x, which passes through LDS in chunks of CH
// steps, two buffers in turn.  (Read from L2 by every wave for itself, x costs
// more than the weights: 65536 x 7168 rows and 16 tokens took 150, 101, 77
// and 68 us with 1, 2, 4 and 8 row tiles to a wave.)  In LDS a fragment is 64
// consecutive 16-byte words, the lanes' own, so its reads have no bank
// conflicts.  A step takes half a cache line of each row, so two steps' loads
// are issued together: apart, the line was fetched twice (65536 x 7168, 16
// tokens, 62 us; two steps ahead, apart, 58; now 55, 4.6 TB/s; 49 with one
// token, 5.1 TB/s, 66 with 32).  What a CU takes in at a time bounds it, 18 KB
// a microsecond: two blocks on one run at half the speed each.
constexpr int ML_W = 8;   // waves

template <int RT, int NT, bool SV, typename OT>
__global__ __launch_bounds__(64 * ML_W) void k_fp4_matvec_lds(const uint16_t* __restrict__ x,
                                                              const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ scale, int T, long long N,
                                                              int K, OT* __restrict__ y) {
  constexpr int D = RT == 1 ? 4 : 2, G = 2, CH = 8 / NT;  // steps the weights' loads run ahead, and come together
  using S = Skinny<MOE_E2M1, uint16_t, RT, NT, SV>;
  constexpr int FRAGS = CH * NT * S::XV, MINE = FRAGS / ML_W;  // fragments of a chunk, and those that a wave stages
  static_assert(FRAGS % ML_W == 0 && CH % D == 0, "chunks are staged by all waves, and are turns of the ring");
  __shared__ sk_u32x4 lds[2][FRAGS][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long row0 = ((long long)blockIdx.x * ML_W + wave) * (16 * RT);
  const int rows = (int)(row0 >= N ? 0 : N - row0 < 16 * RT ? N - row0 : 16 * RT);
  const int t0 = blockIdx.y * (16 * NT);
  const int toks = T - t0 < 16 * NT ? T - t0 : 16 * NT;
  typename S::Lanes L;
  L.K = K;
  L.g = lane >> 4;
  // a wave without rows (all its lanes' offsets are past the end) stages x all
  // the same; its buffers are the matrix's first row
  const long long base = rows > 0 ? row0 : 0;
  const uint32_t held = rows > 0 ? rows : 1;
  L.rw = sk_rsrc(q + base * (K / 2), held * (uint32_t)(K / 2));
  L.rs = sk_rsrc(scale + base * (K / 32), held * (uint32_t)(K / 32));
  L.rx = sk_rsrc(x + (long long)t0 * K, (uint32_t)toks * (uint32_t)K * 2u);
#pragma unroll
  for (int f = 0; f < RT; ++f) {
    const int r = f * 16 + (lane & 15);
    L.w_off[f] = r < rows ? (uint32_t)r * (uint32_t)(K / 2) + L.g * 16u : SK_OOB;
    L.s_off[f] = r < rows ? (uint32_t)r * (uint32_t)(K / 32) + (SV ? 0 : L.g) : SK_OOB;
  }
  const int steps = (K + S::STEP - 1) / S::STEP, chunks = (steps + CH - 1) / CH;
  // fragment i of a chunk: step i / (NT XV), token tile, 16 bytes of the lane's 64
  sk_u32x4 stage[MINE];
  auto fetch = [&](int c) {
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int i = wave * MINE + m;
      const int t = i / S::XV % NT * 16 + (lane & 15), k = (c * CH + i / (NT * S::XV)) * S::STEP + L.g * S::EPL;
      const uint32_t off = t < toks && k < K ? ((uint32_t)t * (uint32_t)K + (uint32_t)k) * 2u : SK_OOB;
      stage[m] = __builtin_amdgcn_raw_buffer_load_b128(L.rx, off, i % S::XV * 16, 0);
    }
  };
  auto put = [&](int c) {
#pragma unroll
    for (int m = 0; m < MINE; ++m) lds[c & 1][wave * MINE + m][lane] = stage[m];
    // the LDS writes alone are waited for: the loads in flight stay so.  One
    // statement, so that no access comes to lie between the wait and the barrier
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  sk_f32x4 acc[RT][NT];
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[f][n] = sk_f32x4{0.f, 0.f, 0.f, 0.f};
  typename S::Step st[D];
  typename S::Scales sc[2];
  fetch(0);
  if (SV) S::load_scales(sc[0], L, 0);
#pragma unroll
  for (int i = 0; i < D; ++i) {
    S::load_w(st[i], L, i);  // past the last step: nothing is fetched
    __builtin_amdgcn_sched_barrier(0);
  }
  put(0);
  for (int c = 0; c < chunks; ++c) {
    if (c + 1 < chunks) fetch(c + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int s = c * CH + i;
      if (SV && i % 4 == 0 && s + 4 < steps) S::load_scales(sc[1], L, s + 4);
      if (s < steps) {  // past it the exponent bytes are the next row's
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int v = 0; v < S::XV; ++v) st[i % D].x[n][0][v] = lds[c & 1][(i * NT + n) * S::XV + v][lane];
        S::mma(acc, st[i % D], L, sc[0], i % 4);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (i % G == G - 1)
#pragma unroll
        for (int j = i - G + 1; j <= i; ++j) S::load_w(st[j % D], L, c * CH + j + D);
      __builtin_amdgcn_sched_barrier(0);
      if (SV && i % 4 == 3) sc[0] = sc[1];
    }
    if (c + 1 < chunks) put(c + 1);
  }
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = n * 16 + (lane & 15), r = f * 16 + 4 * L.g;
      if (t >= toks || r >= rows) continue;
      mv_store(y + (long long)(t0 + t) * N + row0 + r, acc[f][n], rows - r);
    }
}

constexpr int MV_MAX_K = 1 << 20;  // 64 rows and 32 tokens of it stay within 32-bit offsets

}  // namespace

moe_status fp4_quantize(const void* x, moe_dtype x_t, long long rows, long long cols, uint8_t* q, uint8_t* scale,
                        void* stream) {
  MOE_REQUIRE(x_t == MOE_F32 || x_t == MOE_BF16, MOE_EINVAL, "x_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(rows >= 0 && cols >= 0 && cols % 32 == 0, MOE_EINVAL, "cols must be a multiple of 32");
  MOE_REQUIRE(rows == 0 || cols == 0 || (x && q && scale), MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(x) && aligned16(q), MOE_EINVAL, "x and q must be 16-byte aligned");
  MOE_REQUIRE(rows == 0 || cols <= (1LL << 40) / rows, MOE_EINVAL, "too many values");
  const long long chunks = rows * (cols / 8);
  if (chunks == 0) return MOE_OK;
  hipStream_t st = as_stream(stream);
  const dim3 grid(chunk_blocks(chunks));
  if (x_t == MOE_F32)
    hipLaunchKernelGGL(k_fp4_quant<float>, grid, dim3(256), 0, st, static_cast<const float*>(x), chunks, q, scale);
  else
    hipLaunchKernelGGL(k_fp4_quant<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(x), chunks, q, scale);
  return launch_status("fp4_quantize_groups");
}

moe_status fp4_dequantize(const uint8_t* q, const uint8_t* scale, long long rows, long long cols, void* out,
                          moe_dtype out_t, void* stream) {
  MOE_REQUIRE(out_t == MOE_F32 || out_t == MOE_BF16, MOE_EINVAL, "out_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(rows >= 0 && cols >= 0 && cols % 32 == 0, MOE_EINVAL, "cols must be a multiple of 32");
  MOE_REQUIRE(rows == 0 || cols == 0 || (q && scale && out), MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(out), MOE_EINVAL, "q and out must be 16-byte aligned");
  MOE_REQUIRE(rows == 0 || cols <= (1LL << 40) / rows, MOE_EINVAL, "too many values");
  const long long chunks = rows * (cols / 8);
  if (chunks == 0) return MOE_OK;
  hipStream_t st = as_stream(stream);
  const dim3 grid(chunk_blocks(chunks));
  if (out_t == MOE_F32)
    hipLaunchKernelGGL(k_fp4_dequant<float>, grid, dim3(256), 0, st, q, scale, chunks, static_cast<float*>(out));
  else
    hipLaunchKernelGGL(k_fp4_dequant<uint16_t>, grid, dim3(256), 0, st, q, scale, chunks, static_cast<uint16_t*>(out));
  return launch_status("fp4_dequantize_groups");
}

moe_status fp4_matvec(const void* x, moe_dtype x_t, const uint8_t* q, const uint8_t* scale, int T, long long N, int K,
                      void* y, moe_dtype y_t, void* stream) {
  MOE_REQUIRE(x_t == MOE_F32 || x_t == MOE_BF16, MOE_EINVAL, "x_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(y_t == MOE_F32 || y_t == MOE_BF16, MOE_EINVAL, "y_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(x_t == MOE_BF16, MOE_EUNSUPPORTED, "x must be bf16");
  MOE_REQUIRE(T >= 0 && N >= 0 && K >= 32 && K % 32 == 0, MOE_EINVAL,
              "need T, N >= 0 and K a positive multiple of 32");
  MOE_REQUIRE(K <= MV_MAX_K, MOE_EUNSUPPORTED, "K above 1048576");
  // 16 threads to a row at most: a launch has fewer than 2^32
  MOE_REQUIRE(T <= 16 * 65535 && N <= (1LL << 27), MOE_EUNSUPPORTED, "T above 1048560 or N above 2^27");
  if (T == 0 || N == 0) return MOE_OK;
  MOE_REQUIRE(x && q && scale && y, MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(x) && aligned16(q), MOE_EINVAL, "x and q must be 16-byte aligned");
  hipStream_t st = as_stream(stream);
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  // rows, tokens of a block
  auto go = [&](auto kernel, int waves, int rows, int tokens, auto* out) {
    const dim3 grid((unsigned)ceil_div(N, rows), (unsigned)ceil_div(T, tokens));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), 0, st, xb, q, scale, T, N, K, out);
  };
  // In us, K = 7168 (the limits hold for every K; at others they were not
  // measured; up to 16384 rows the weights came from the last-level cache, from
  // memory these calls take up to a quarter longer).  Through LDS a CU takes 128 rows at a time in about 27 (up
  // to 16 tokens; 32 tokens 34) and 256 in twice that, however many of its
  // neighbours have none left: `units` of 32768 rows, with one row tile to a wave
  // when their number is odd (81920 rows, 16 tokens, 86, with two tiles 105), else
  // two (65536: 55 / 60; 131072: 118 / 120).  The other form takes 40 a unit (32
  // tokens 55), up to 4 tokens packed 27 to 31, of the rows there are: LDS where
  // enough of the last unit is filled (32768 rows, one token 28 / 30, 4 tokens 29 /
  // 33, 16 tokens 33 / 40; 65536: 49 / 53, 52 / 62, 55 / 81; 100003, 2 tokens:
  // 95 / 87).
  // Below that, rows to a block, up to 4 tokens, packed, 1 and 4 tokens: 4096
  // rows 6.0 / 6.1 with one row tile, 7.8 / 7.9 with two (not packed 6.6 / 7.6);
  // 16384: 12.8 / 13.3, two 13.4 / 13.4; 32768: 31 / 35, two 28 / 31.  16 and 32
  // tokens: 4096 rows, one tile 11 / 17, two 13 / 19; 8192: two 13 / 19, one 18 /
  // 30, four 17 / 23; 16384: four 18 / 25, two 22 / 37, LDS 23 / 32.
  const long long units = ceil_div(N, 32768);
  const bool lds = N * 16 >= units * 32768 * (T > 4 ? 11 : 14);
  auto shape = [&](auto sv, auto* out) {
    constexpr bool SV = decltype(sv)::value;
    using OT = std::remove_pointer_t<decltype(out)>;
    auto many = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      if (lds && units % 2 == 0)
        go(k_fp4_matvec_lds<2, NT, SV, OT>, ML_W, 32 * ML_W, 16 * NT, out);
      else if (lds)
        go(k_fp4_matvec_lds<1, NT, SV, OT>, ML_W, 16 * ML_W, 16 * NT, out);
      else if (N >= 12288)
        go(k_fp4_matvec<4, NT, SV, false, OT>, MV_W, 64, 16 * NT, out);
      else if (N >= 6144)
        go(k_fp4_matvec<2, NT, SV, false, OT>, MV_W, 32, 16 * NT, out);
      else
        go(k_fp4_matvec<1, NT, SV, false, OT>, MV_W, 16, 16 * NT, out);
    };
    if (T > 16)
      many(std::integral_constant<int, 2>{});
    else if (T > 4 || lds)
      many(std::integral_constant<int, 1>{});
    else if (N >= 24576)
      go(k_fp4_matvec<2, 1, SV, true, OT>, MV_W, 32, 4, out);
    else
      go(k_fp4_matvec<1, 1, SV, true, OT>, MV_W, 16, 4, out);
  };
  // rows of exponent bytes in whole words: read 16 at a time
  const bool words = K % 128 == 0 && aligned4(scale);
  auto pick = [&](auto* out) {
    if (words) shape(std::true_type{}, out); else shape(std::false_type{}, out);
  };
  if (y_t == MOE_BF16) pick(static_cast<uint16_t*>(y)); else pick(static_cast<float*>(y));
  return launch_status("fp4_matvec");
}

}  // namespace moe
