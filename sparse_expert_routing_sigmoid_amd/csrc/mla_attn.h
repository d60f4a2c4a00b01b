// What the expanded attention and its gradient share: the arguments, a
// block's place among the packed sequences, and the staged tiles of 64 keys.
#pragma once

#include "mla.h"

namespace moe {

constexpr int ATTN_MAX_B = 8192;
constexpr long long ATTN_MAX_TILES = 1LL << 22;

struct AttnArgs {
  const uint16_t *q, *kv, *k_rope;
  long long ldr;  // elements from one token's k_rope to the next
  const int32_t *cu_q, *cu_k;
  int B;
  long long Tq, Tk;
  int H, dn, dr, dv;
  bool causal;
  float scale;
  int rows;            // of a block's tile
  bool by_key;         // the tiles are of keys
  long long tiles;     // a bound on the tiles of all sequences: each begins its own
  long long per_xcd;   // blocks an XCD
};

inline moe_status attn_check(const char* where, const void* q, const void* kv, const void* k_rope, long long ldr,
                             const int32_t* cu_q, const int32_t* cu_k, int B, long long Tq, long long Tk, int H, int dn,
                             int dr, int dv, float scale) {
  auto bad = [&](moe_status st, const char* msg) {
    set_error(std::string(where) + ": " + msg);
    return st;
  };
  if (!(B >= 0 && Tq >= 0 && Tk >= 0 && Tq < (1LL << 31) && Tk < (1LL << 31) && H >= 1))
    return bad(MOE_EINVAL, "need B >= 0, 0 <= Tq, Tk < 2^31 and H >= 1");
  if (!(dn >= 8 && dr >= 8 && dv >= 8 && dn % 8 == 0 && dr % 8 == 0 && dv % 8 == 0))
    return bad(MOE_EINVAL, "dn, dr and dv must be positive multiples of 8");
  if (!mla_dims_ok(dn, dr, dv)) return bad(MOE_EUNSUPPORTED, "dn or dv above 128, or dr above 64");
  if (B > ATTN_MAX_B) return bad(MOE_EUNSUPPORTED, "more sequences than MLA_MAX_REQUESTS");
  if (H > 1024) return bad(MOE_EUNSUPPORTED, "more than 1024 heads");
  // the grids stay below 2^32 threads: tiles of 128 rows, 512 threads; dk_rope by 4 values a thread
  const long long tiles = (Tq > Tk ? Tq : Tk) / 128 + B;
  if (tiles * H > ATTN_MAX_TILES || Tk * dr > (1LL << 33))
    return bad(MOE_EUNSUPPORTED, "more than 2^22 tiles of 128 rows and a head, or 2^33 values in k_rope");
  if (!mla_scale_ok(scale)) return bad(MOE_EINVAL, "scale must be positive and at most 2^127");
  if (!(ldr >= dr && ldr % 8 == 0 && ldr <= (1 << 20)))
    return bad(MOE_EINVAL, "k_rope's row stride must be a multiple of 8 that holds a row, at most 2^20");
  if (Tq > 0 && B > 0 && !(q && cu_q && cu_k && (Tk == 0 || (kv && k_rope)))) return bad(MOE_EINVAL, "NULL pointer");
  if (!(aligned16(q) && aligned16(kv) && aligned16(k_rope)))
    return bad(MOE_EINVAL, "q, kv and k_rope must be 16-byte aligned");
  return MOE_OK;
}

// Tiles of `rows` of T query or key rows; the grid gives each of the 8 XCDs
// (block b runs on XCD b % 8) a run of (head, tile) pairs, so that a head's
// keys meet in one L2.
inline AttnArgs attn_args(const void* q, const void* kv, const void* k_rope, long long ldr, const int32_t* cu_q,
                          const int32_t* cu_k, int B, long long Tq, long long Tk, int H, int dn, int dr, int dv,
                          bool causal, float scale, int rows, bool by_key) {
  const long long T = by_key ? Tk : Tq;
  const long long tiles = T / rows + (B < T ? B : T);
  return {static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(kv), static_cast<const uint16_t*>(k_rope), ldr,
          cu_q, cu_k, B, Tq, Tk, H, dn, dr, dv, causal, scale, rows, by_key, tiles, ceil_div(tiles * H, 8)};
}

struct AttnTile {
  long long q0, k0;  // first rows of the sequence
  int lq, lk;
  int row0;  // first row of the tile within the sequence; -1: no tile
};

// The tile of this block.  Tiles are numbered through the sequences; of a
// head's query tiles the last come first (under a causal mask they see the most
// keys), of its key tiles the first.
// Every thread counts the tiles of a run of sequences, a scan places the runs,
// and the owner of the tile walks its run.  Lengths are taken from cu clamped
// to the rows there are, so no offsets lead outside the tensors.
// `lds` is lent for the while.
template <int WAVES = 4>
__device__ __forceinline__ AttnTile attn_find(const AttnArgs& a, int& h, uint8_t* lds) {
  long long* sum = reinterpret_cast<long long*>(lds);
  AttnTile& found = *reinterpret_cast<AttnTile*>(lds + 128);
  const long long item = (blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  AttnTile none{0, 0, 0, 0, -1};
  h = 0;
  if (item >= a.tiles * a.H) return none;
  h = (int)(item / a.tiles);
  const long long nth = item - (long long)h * a.tiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (a.B + 64 * WAVES - 1) / (64 * WAVES), b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  auto at = [](const int32_t* cu, int b, long long T) { return min(max((long long)cu[b], 0LL), T); };
  const int32_t* cu = a.by_key ? a.cu_k : a.cu_q;
  const long long T = a.by_key ? a.Tk : a.Tq;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const long long n = at(cu, b + 1, T) - at(cu, b, T);
    mine += n > 0 ? (n + a.rows - 1) / a.rows : 0;
  }
  long long s = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long long t = __shfl_up(s, off, 64);
    if (lane >= off) s += t;
  }
  if (lane == 63) sum[wave] = s;
  if (threadIdx.x == 0) found.row0 = -1;
  __syncthreads();
  long long before = s - mine, total = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    if (i < wave) before += sum[i];
    total += sum[i];
  }
  const long long want = a.by_key ? nth : total - 1 - nth;
  if (want >= before && want < before + mine) {
    long long first = before;
    for (int b = b0; b < b1; ++b) {
      const long long lo = at(cu, b, T), n = at(cu, b + 1, T) - lo;
      const long long here = n > 0 ? (n + a.rows - 1) / a.rows : 0;
      if (want < first + here) {
        AttnTile f;
        f.q0 = at(a.cu_q, b, a.Tq);
        f.k0 = at(a.cu_k, b, a.Tk);
        f.lq = (int)max(0LL, at(a.cu_q, b + 1, a.Tq) - f.q0);
        f.lk = (int)max(0LL, at(a.cu_k, b + 1, a.Tk) - f.k0);
        f.row0 = (int)(want - first) * a.rows;
        found = f;
        break;
      }
      first += here;
    }
  }
  __syncthreads();
  AttnTile f = found;
  __syncthreads();
  // the same in every lane: kept in scalar registers
  f.row0 = __builtin_amdgcn_readfirstlane(f.row0);
  f.lq = __builtin_amdgcn_readfirstlane(f.lq);
  f.lk = __builtin_amdgcn_readfirstlane(f.lk);
  f.q0 = __builtin_amdgcn_readfirstlane((int)f.q0);
  f.k0 = __builtin_amdgcn_readfirstlane((int)f.k0);
  return f;
}

// Rows of one array staged in LDS with CPR chunks each: `first` is the offset
// of this thread's first chunk from the tile's first row, OOB for a chunk past
// the array's columns.  Later chunks lie a fixed number of rows below, whose
// swizzle is the same (a multiple of 16).  Where a tile has fewer chunks than
// the block has threads, waves load the same ones twice.
template <int CPR, int ROWS, int BLOCK = 4>  // BLOCK: waves of the block
struct RowStage {
  static constexpr int CHUNKS = ROWS * CPR, WAVES = CHUNKS < 64 * BLOCK ? CHUNKS / 64 : BLOCK;
  static constexpr int BYTES = CHUNKS * 16, LOADS = CHUNKS / (64 * WAVES), STEP = 64 * WAVES / CPR;
  static_assert(CHUNKS % (64 * WAVES) == 0 && (LOADS == 1 || STEP % 16 == 0), "");
  uint32_t first, step;
  __device__ __forceinline__ void init(uint32_t row_bytes, int cols, int lane, int wave) {
    const int p = wave % WAVES * 64 + lane, r = p / CPR, c = (p % CPR) ^ swz<CPR>(r);
    first = 8 * c < cols ? r * row_bytes + 16 * c : MLA_OOB;
    step = STEP * row_bytes;
  }
  __device__ __forceinline__ void load(int j, uint8_t* lds, __amdgpu_buffer_rsrc_t r, int wave) const {
    mla_dma16(r, lds + (WAVES * j + wave % WAVES) * 1024, first + j * step);
  }
};

// KEYS keys of one head: k^n, r and v, each rows of its own.  The buffer of a
// load ends with the sequence's last row, so later rows read as zeros.  aim()
// names a tile and its place, load() issues one of its LOADS loads: they go out
// between products.
template <int DN, int DR, int DV, int KEYS = 64>
struct KeyTile {
  static constexpr int CN = DN / 8, CR = DR / 8, CV = DV / 8;
  static constexpr int KN = KEYS * DN * 2, KR = KEYS * DR * 2, V = KEYS * DV * 2, BYTES = KN + KR + V;
  typedef RowStage<CN, KEYS> SN;
  typedef RowStage<CR, KEYS> SR;
  typedef RowStage<CV, KEYS> SV;
  static constexpr int LOADS = SN::LOADS + SR::LOADS + SV::LOADS;
  SN sn;
  SR sr;
  SV sv;
  const uint16_t *kv, *rope;
  uint32_t kv_row, rope_row;
  int rows, dn, dr, dv, wave;
  uint8_t* to;
  __amdgpu_buffer_rsrc_t rn, rr, rv;
  // `rows`: the keys that any query of the block sees
  __device__ __forceinline__ void init(const AttnArgs& a, int h, long long k0, int rows_, int lane, int wave_) {
    kv_row = (uint32_t)a.H * (a.dn + a.dv) * 2;
    rope_row = (uint32_t)a.ldr * 2;
    kv = a.kv + (k0 * a.H + h) * (a.dn + a.dv);
    rope = a.k_rope + k0 * a.ldr;
    rows = rows_, dn = a.dn, dr = a.dr, dv = a.dv, wave = wave_;
    sn.init(kv_row, dn, lane, wave_);
    sr.init(rope_row, dr, lane, wave_);
    sv.init(kv_row, dv, lane, wave_);
  }
  __device__ __forceinline__ void aim(uint8_t* lds, int t) {
    const int n = min(KEYS, rows - KEYS * t) - 1;  // the last row of the tile; below 0: no rows, and nothing is read
    const uint16_t* b = kv + (n < 0 ? 0 : (long long)t * KEYS * (kv_row / 2));
    const uint16_t* r = rope + (n < 0 ? 0 : (long long)t * KEYS * (rope_row / 2));
    to = lds;
    rn = mla_rsrc(b, n < 0 ? 0 : n * kv_row + dn * 2);
    rr = mla_rsrc(r, n < 0 ? 0 : n * rope_row + dr * 2);
    rv = mla_rsrc(b + dn, n < 0 ? 0 : n * kv_row + dv * 2);
  }
  __device__ __forceinline__ void load(int j) const {
    if (j < SN::LOADS)
      sn.load(j, to, rn, wave);
    else if (j < SN::LOADS + SR::LOADS)
      sr.load(j - SN::LOADS, to + KN, rr, wave);
    else if (j < LOADS)
      sv.load(j - SN::LOADS - SR::LOADS, to + KN + KR, rv, wave);
  }
  __device__ __forceinline__ void load_all(uint8_t* lds, int t) {
    aim(lds, t);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load(j);
  }
};

// 32 queries of one head: q^n, q^r and the gradient of their outputs, and lse
// (in powers of two) and D of each.
template <int DN, int DR, int DV>
struct QueryTile {
  static constexpr int ROWS = 32, CN = DN / 8, CR = DR / 8, CV = DV / 8;
  static constexpr int QN = ROWS * DN * 2, QR = ROWS * DR * 2, DO = ROWS * DV * 2, BYTES = QN + QR + DO + 8 * ROWS;
  typedef RowStage<CN, ROWS, 8> SN;
  typedef RowStage<CR, ROWS, 8> SR;
  typedef RowStage<CV, ROWS, 8> SO;
  static constexpr int LOADS = SN::LOADS + SR::LOADS + SO::LOADS + 1;
  SN sn;
  SR sr;
  SO so;
  const uint16_t *q, *dout;
  const float* stat;
  uint32_t q_row, o_row, one;
  int lq, dn, dr, dv, H, wave;
  uint8_t* to;
  __amdgpu_buffer_rsrc_t rn, rr, ro, rl;
  __device__ __forceinline__ void init(const AttnArgs& a, const uint16_t* dout_, const float* stat_, int h, long long q0,
                                       int lq_, int lane, int wave_) {
    q_row = (uint32_t)a.H * (a.dn + a.dr) * 2;
    o_row = (uint32_t)a.H * a.dv * 2;
    q = a.q + (q0 * a.H + h) * (a.dn + a.dr);
    dout = dout_ + (q0 * a.H + h) * a.dv;
    stat = stat_ + (q0 * a.H + h) * 2;
    lq = lq_, dn = a.dn, dr = a.dr, dv = a.dv, H = a.H, wave = wave_;
    one = (uint32_t)(lane & 31) * a.H * 8 + (lane >> 5) * 4;
    sn.init(q_row, dn, lane, wave_);
    sr.init(q_row, dr, lane, wave_);
    so.init(o_row, dv, lane, wave_);
  }
  __device__ __forceinline__ void aim(uint8_t* lds, int t) {
    const int n = min(ROWS, lq - ROWS * t) - 1;  // the last row of the tile; below 0: no rows, and nothing is read
    const long long at = n < 0 ? 0 : t * ROWS;
    const uint16_t* b = q + at * (q_row / 2);
    to = lds;
    rn = mla_rsrc(b, n < 0 ? 0 : n * q_row + dn * 2);
    rr = mla_rsrc(b + dn, n < 0 ? 0 : n * q_row + dr * 2);
    ro = mla_rsrc(dout + at * (o_row / 2), n < 0 ? 0 : n * o_row + dv * 2);
    rl = mla_rsrc(stat + at * H * 2, n < 0 ? 0 : n * H * 8 + 8);
  }
  __device__ __forceinline__ void load(int j) const {
    if (j < SN::LOADS)
      sn.load(j, to, rn, wave);
    else if (j < SN::LOADS + SR::LOADS)
      sr.load(j - SN::LOADS, to + QN, rr, wave);
    else if (j < LOADS - 1)
      so.load(j - SN::LOADS - SR::LOADS, to + QN + QR, ro, wave);
    else if (j == LOADS - 1)  // every wave the same
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rl, (lds_void*)(to + QN + QR + DO), 4, one, 0, 0, 0);
  }
  __device__ __forceinline__ void load_all(uint8_t* lds, int t) {
    aim(lds, t);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load(j);
  }
};

}  // namespace moe
