// Shared device pieces of the latent attention kernels: tiles of rows staged
// in LDS, the two ways their fragments are read, and packing.
//
// A tile holds rows of CPR 16-byte chunks as they lie in memory, chunk c of
// row r at chunk c ^ swz<CPR>(r).  It is read
//   by rows (frag_row): a lane gets 8 consecutive values of its row, the
//     operand of v_mfma_f32_32x32x16_bf16 whose K axis is the row's;
//   by columns (frag_tr): a lane gets 8 rows' values of its column, by two
//     transposing reads (in a group of 16 lanes, lane j names row j / 4 and
//     columns 4 (j % 4) .. + 3 and lane i receives column i of the 4 rows).
// A 32x32 result tile leaves lane l with column l % 32 and rows 8 (r / 4) +
// 4 (l / 32) + r % 4 in register r.  Packed in pairs, registers 8 i .. 8 i + 7
// are an operand for the next product's K step i whose K order is that of the
// rows; frag_tr reads in the same order, so scores never move between lanes.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;

constexpr int MLA_MAX_DN = 128, MLA_MAX_DR = 64, MLA_MAX_DV = 128, MLA_MAX_DC = 512;
constexpr uint32_t MLA_OOB = 0x80000000u;  // an offset past every buffer: the load writes zeros
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

inline bool mla_dims_ok(int dn, int dr, int dv) {
  return dn >= 8 && dn % 8 == 0 && dn <= MLA_MAX_DN && dr >= 8 && dr % 8 == 0 && dr <= MLA_MAX_DR && dv >= 8 &&
         dv % 8 == 0 && dv <= MLA_MAX_DV;
}
inline bool mla_scale_ok(float scale) { return scale > 0.f && scale <= 0x1p127f; }  // scale * LOG2E is finite
inline bool mla_dc_ok(int dc) { return dc >= 8 && dc % 8 == 0 && dc <= MLA_MAX_DC; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mla_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Lane l writes LDS bytes [16 l, 16 l + 16) of the 1 KB block at `lds`.
__device__ __forceinline__ void mla_dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, 0, 0, 0);
}

// s_waitcnt's operand for no vector memory access in flight (expcnt and lgkmcnt
// at their maxima).
constexpr int WAIT_VM0 = (7 << 4) | (15 << 8);

// Every load into LDS of this wave has landed, its LDS reads are done, and so
// are the other waves'.
__device__ __forceinline__ void mla_sync() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The same for LDS accesses alone: loads stay in flight.
__device__ __forceinline__ void mla_sync_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Rows that one wave instruction touches fall on distinct banks: 16 rows of
// one chunk (frag_row), and 4 rows of 4 chunks (frag_tr), over 128 bytes a
// cycle or 256.
template <int CPR>
__host__ __device__ constexpr int swz(int r) {
  const int y = r & 3, z = (r >> 2) & 3;
  return CPR >= 16 ? ((4 * y + 2 * ((y ^ (y >> 1)) & 1)) ^ z) : CPR == 8 ? ((2 * y) ^ z) : z;
}

// A value from or to LDS that no direct-to-LDS load writes.  The restrict
// parameter gives the access an alias scope that those loads do not share:
// without it the compiler waits here for every such load in flight.
template <typename V>
__device__ __forceinline__ V lds_get(const void* __restrict__ p) {
  return *static_cast<const V*>(p);
}

template <typename V>
__device__ __forceinline__ void lds_put(void* __restrict__ p, V v) {
  *static_cast<V*>(p) = v;
}

// A lane's share of the fragment addresses in a tile: chunk 0 of its row, and
// its place in a transposing read of columns 0 and rows 0.  The rest of an
// address is a XOR of chunk bits and a constant.  fresh() gives values that
// the compiler can't carry across a loop: kept there, the addresses of all
// fragments would take the registers that the sums need.
template <int CPR>
struct FragAt {
  uint32_t row, tr;
  __device__ __forceinline__ explicit FragAt(int lane) {
    const int r = lane & 31, g = lane >> 4, k = 4 * (g >> 1) + ((lane & 15) >> 2);
    row = r * CPR * 16 + (((lane >> 5) ^ swz<CPR>(r)) << 4);
    tr = k * CPR * 16 + (((2 * (g & 1) + ((lane & 3) >> 1)) ^ swz<CPR>(k)) << 4) + (lane & 1) * 8;
  }
  __device__ __forceinline__ FragAt fresh() const {
    FragAt f = *this;
    asm volatile("" : "+v"(f.row), "+v"(f.tr));
    return f;
  }
};

// Rows r0 + l % 32, values 16 ks + 8 (l / 32) .. + 7 (r0 % 16 == 0).
template <int CPR>
__device__ __forceinline__ bf16x8_t frag_row(const uint8_t* __restrict__ t, FragAt<CPR> at, int r0, int ks) {
  return __builtin_bit_cast(
      bf16x8_t, *reinterpret_cast<const u32x4_t*>(t + (at.row ^ ((ks & 7) << 5)) + (r0 * CPR * 16 + (ks >> 3) * 256)));
}

// Columns 32 d + l % 32, rows k0 + 8 (e / 4) + 4 (l / 32) + e % 4, e = 0..7
// (k0 % 16 == 0).  The restrict parameter: as in lds_get.
template <int CPR>
__device__ __forceinline__ bf16x8_t frag_tr(const uint8_t* __restrict__ t, FragAt<CPR> at, int k0, int d) {
  const int by = k0 * CPR * 16 + (d >> 2) * 256;
  const uint8_t* p0 = t + (at.tr ^ ((d & 3) << 6)) + by;
  const uint8_t* p1 = t + (at.tr ^ ((d & 3) << 6) ^ ((swz<CPR>(0) ^ swz<CPR>(8)) << 4)) + (by + 8 * CPR * 16);
  const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p0);
  const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p1);
  const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// Values i .. i + 7 of a result tile as a K step's operand.
__device__ __forceinline__ bf16x8_t pack8(const f32x16_t& v, int i) {
  const u32x4_t w = {pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]), pack_bf16x2(v[i + 4], v[i + 5]),
                     pack_bf16x2(v[i + 6], v[i + 7])};
  return __builtin_bit_cast(bf16x8_t, w);
}

__device__ __forceinline__ f32x16_t mma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16_t zero16() {
  f32x16_t z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// 16 bytes of bf16 at p[at], or zeros (p[0] is read then, so a run of loads
// has no branches and waits once).
__device__ __forceinline__ bf16x8_t load8(const uint16_t* p, int at, bool live) {
  u32x4_t v = *reinterpret_cast<const u32x4_t*>(p + (live ? at : 0));
  const u32x4_t z = {0, 0, 0, 0};
  return __builtin_bit_cast(bf16x8_t, live ? v : z);
}

// N products, use(i, load(i)), with the LDS reads of the AHEAD next ones under
// way at each: begun by start() and kept in the order that is written, but for
// arithmetic.  (Left to itself the compiler, sparing registers, puts each read
// right before its use, and a lone wave waits out the LDS latency at every
// product.)
template <int N, int AHEAD>
struct Ahead {
  bf16x8_t f[AHEAD];
  template <typename L>
  __device__ __forceinline__ void start(L load) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) f[i] = load(i);
    __builtin_amdgcn_sched_barrier(0x6);
  }
  template <int FROM = 0, int TO = N, typename L, typename U>
  __device__ __forceinline__ void run(L load, U use) {
#pragma unroll
    for (int i = FROM; i < TO; ++i) {
      use(i, f[i % AHEAD]);
      if (i + AHEAD < N) f[i % AHEAD] = load(i + AHEAD);
      __builtin_amdgcn_sched_barrier(0x6);
    }
  }
};

// The larger, and the sum, of a column's two halves, in both lanes that hold it.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Whether c holds in any lane; the same for the whole wave, which the compiler
// can tell.
__device__ __forceinline__ bool wave_any(bool c) { return __builtin_amdgcn_ballot_w64(c) != 0; }

// The reference point m of a running softmax (in powers of two), moved up to
// the new scores' maximum where one passes it by more than 8: weights then stay
// below 2^8, the sums l and o carry them as well as weights below 1, and the
// sums are rescaled a few times a row instead of at every tile.
template <int N>
__device__ __forceinline__ void rescale(float& m, float& l, f32x16_t (&o)[N], float top) {
  if (!wave_any(top > m + 8.f)) return;
  const float mn = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
  m = mn;
  l *= f;
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[d][r] *= f;
}

// Four consecutive fp32 results, as fp32 or rounded to bf16.
__device__ __forceinline__ void store4(void* p, long long at, bool bf16, float a, float b, float c, float d) {
  if (bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(a, b, c, d);
}

// A result tile times f to 32 columns of this lane's row at p[at], those below
// `cols`.  For bf16 the two lanes of a row trade halves of every other 8 columns,
// so that each stores 16 bytes: stores of rows that lie apart take a turn of the
// memory pipe for each lane, whatever their size (the gradient of 16 sequences of
// 100, 16 heads: 57.3 -> 53.6 us).
__device__ __forceinline__ void store_tile(void* p, long long at, bool bf16, const f32x16_t& v, float f, int half,
                                           int cols) {
  if (bf16) {
#pragma unroll
    for (int r = 0; r < 16; r += 8) {
      const auto x = __builtin_amdgcn_permlane32_swap(pack_bf16x2(v[r] * f, v[r + 1] * f),
                                                      pack_bf16x2(v[r + 4] * f, v[r + 5] * f), false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(pack_bf16x2(v[r + 2] * f, v[r + 3] * f),
                                                      pack_bf16x2(v[r + 6] * f, v[r + 7] * f), false, false);
      const int c = 2 * r + 8 * half;
      if (c < cols)
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + at + c) = u32x4_t{x[0], y[0], x[1], y[1]};
    }
  } else {
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int c = 2 * r + 4 * half;
      if (c < cols) store4(p, at + c, false, v[r] * f, v[r + 1] * f, v[r + 2] * f, v[r + 3] * f);
    }
  }
}

}  // namespace moe
