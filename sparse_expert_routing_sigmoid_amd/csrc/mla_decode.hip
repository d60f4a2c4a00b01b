// Latent attention of the newest S tokens of each request over the paged
// cache, in absorbed form.  With k_{j,h} = [W^K_h c_j ; r_j], v_{j,h} = W^V_h c_j:
//   q~_h = (W^K_h)^T q^n_h,  s_j = scale (q~_h . c_j + q^r_h . r_j)
//   o~_h = sum_j softmax(s)_j c_j,  o_h = W^V_h o~_h
// so that all heads read the same dc + dr values of a cached token.
//
// k_absorb forms q~, rounded to bf16 as an operand of the next product: 2^-8 of a
// value at most, of either sign, so a score is off by some 2^-9 of the size of its
// c part, as it is where k is rounded in the expanded form.  (A second half of q~
// for blocks of 32 rows, whose registers hold it, took 24 % more time at 31
// requests of 6000 tokens and 14 % at one of 200: not kept.)  The softmax weights
// are rounded likewise for their product where a block has 64 rows, whose
// registers and LDS are full; with 32 rows they pass in two halves, 2^-16 of a
// weight, for at most 4 % of the time (one request of 200 tokens, 8 heads: bf16
// outputs 0.0023 of the norm from exact ones instead of 0.0025, of which their own
// rounding is 0.0017).  Their sum is that of the unrounded ones.
// k_decode: the tiles of 64 tokens of all requests are numbered through, and
// each of `workers` runs takes an equal share of them, whatever the lengths
// (read on the device, so a captured call follows them); a run that crosses
// requests leaves a piece for each.  A piece is o~ before division, the maximum
// and the sum of its scores for each row (a row is a query token and head).
// k_out joins a row's pieces and multiplies o~, in two bf16 halves, by W^V.
//
// S^T = C Q~^T and O~^T = C^T P^T both read the staged rows of the cache
// (mla.h), which are read from memory once for 32 RG rows.
//
// With work for every CU k_decode's time is a start, a visit of a tile by every CU
// at once so many times, and the requests that a run crosses into.  32 rows: 17 us
// to start (the first loads and q~ behind the search for the request, two more
// barriers in the first tile, the piece's stores), 2.45 a visit where the rows come
// from the last-level cache and 3.3 where they come from memory (302 MB at 5.8
// TB/s), 8.5 for a crossing (loads, q~ and stores once more, nothing under them).  64
// rows: 21, 2.05 (2.2 to 2.8 in a large batch, whose tiles a block for each 64 rows
// visits, the second out of the L2) and 9; the products alone take 1.9 of a visit.
// Measured (k_absorb + k_decode + k_out, us): one request of 200 tokens, 8 heads: 3
// + 11 + 8.5; one of 131072, 128 heads: 5 + 57 + 14; 31 of about 6000, 8 heads, 4
// tokens each: 5 + 54 + 11 (a start, ten more visits and a crossing); 128 of about
// 8000, 128 heads: 13 + 358 + 27.
#include <type_traits>

#include "mla.h"

namespace moe {

namespace {

typedef const __attribute__((address_space(4))) int32_t const_i32;  // read by scalar loads

constexpr int DEC_MAX_B = 8192, DEC_TILE = 64, DEC_CUS = 256;
constexpr long long DEC_MAX_ROWS = 1LL << 26;  // B S H: k_absorb's grid stays below 2^32 threads
// Tiles are rounded up and loads run two halves ahead, 190 tokens past a request's
// last at most: numbers of tokens then stay in 31 bits.
constexpr long long DEC_MAX_LEN = (1LL << 31) - 256;

struct DecArgs {
  const uint16_t *q, *w, *cache;
  const int32_t *table, *seq_len;
  int B, S, H, dn, dr, dv, dc, W, P;
  uint32_t n_pages;
  float scale;
  int workers, row_blocks;
  uint32_t inv_P;  // 2^32 / P, at most 2^32 - 1: j inv_P / 2^32 is j / P or one less
  // workspace
  uint16_t* qa;        // [B S, H, dc] q~
  float* o;            // [workers + B, S H, dc]
  float* ml;           // [workers + B, S H, 2]
  long long* first;    // [B + 1] tiles before each request
};

__device__ __forceinline__ int dec_len(const DecArgs& a, int seq) {
  return min(max(seq, 0), (int)min((long long)a.W * a.P, DEC_MAX_LEN));
}

// Of G workers (as many as there are tiles, at most), w takes tiles
// [w T / G, (w + 1) T / G): at least one, so each leaves its pieces.
__device__ __forceinline__ int dec_workers(const DecArgs& a, long long T) { return (int)min((long long)a.workers, T); }
__device__ __forceinline__ int dec_worker(long long t, long long T, int G) { return (int)(((t + 1) * G - 1) / T); }

// q~ for 32 tokens, a head and 128 columns; block 0 also numbers the tiles.  128
// tokens of 128 heads: 13 us, of which 51 MB from and to memory take 10.5 at a
// copy's rate.  8-byte accesses to q and q~, whose rows 16 apart share their banks,
// conflict (39 % of the LDS cycles).
__global__ __launch_bounds__(256) void k_absorb(DecArgs a) {
  __shared__ __align__(16) uint8_t lds[128 * 256 + 32 * 256];
  __shared__ long long sum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
  const int col_tiles = (a.dc + 127) / 128, N = a.B * a.S;
  const int ct = blockIdx.x % col_tiles, h = blockIdx.x / col_tiles % a.H, n0 = blockIdx.x / col_tiles / a.H * 32;
  if (blockIdx.x == 0) {
    const int per = (a.B + 255) / 256, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += (dec_len(a, a.seq_len[b]) + DEC_TILE - 1) / DEC_TILE;
    long long s = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const long long t = __shfl_up(s, off, 64);
      if (lane >= off) s += t;
    }
    if (lane == 63) sum[wave] = s;
    __syncthreads();
    long long at = s - mine, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < wave) at += sum[i];
      total += sum[i];
    }
    for (int b = b0; b < b1; ++b) {
      a.first[b] = at;
      at += (dec_len(a, a.seq_len[b]) + DEC_TILE - 1) / DEC_TILE;
    }
    if (tid == 0) a.first[a.B] = total;
  }
  // W^K of the head: rows j < dn, columns of this tile
  const uint16_t* w = a.w + (long long)h * (a.dn + a.dv) * a.dc;
  const __amdgpu_buffer_rsrc_t rs = mla_rsrc(w, (uint32_t)a.dn * a.dc * 2);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = (4 * j + wave) * 4 + lane / 16, c = (lane & 15) ^ swz<16>(r);
    mla_dma16(rs, lds + (4 * j + wave) * 1024, 128 * ct + 8 * c < a.dc ? (r * a.dc + 128 * ct + 8 * c) * 2 : MLA_OOB);
  }
  // q^n of the tokens, beside it
  uint8_t* qs = lds + 128 * 256;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = (4 * j + wave) * 4 + lane / 16, c = (lane & 15) ^ swz<16>(t);
    mla_dma16(mla_rsrc(a.q + ((long long)n0 * a.H + h) * (a.dn + a.dr), 0x7FFFFFFF),
              qs + (4 * j + wave) * 1024,
              8 * c < a.dn && n0 + t < N ? (uint32_t)t * a.H * (a.dn + a.dr) * 2 + 16 * c : MLA_OOB);
  }
  mla_sync();
  f32x16_t o = zero16();
  FragAt<16> at(lane);
  at.tr ^= wave << 6;
  const uint8_t* qt = qs + (lane & 31) * 256 + half * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // the K order of frag_tr: rows 8 (e / 4) + 4 half + e % 4 of each 16
    const int sw = swz<16>(lane & 31);
    const i16x4_t lo = *reinterpret_cast<const i16x4_t*>(qt + (((2 * k) ^ sw) << 4));
    const i16x4_t hi = *reinterpret_cast<const i16x4_t*>(qt + (((2 * k + 1) ^ sw) << 4));
    const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    o = mma(frag_tr(lds, at, 16 * k, 0), __builtin_bit_cast(bf16x8_t, v), o);
  }
  // through LDS, so that a token's 128 columns leave as 256 consecutive bytes
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 16; r += 4)
    *reinterpret_cast<uint2*>(lds + (lane & 31) * 272 + (32 * wave + 2 * r + 4 * half) * 2) =
        make_uint2(pack_bf16x2(o[r], o[r + 1]), pack_bf16x2(o[r + 2], o[r + 3]));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 16 * i + tid / 16, c = 128 * ct + 8 * (tid & 15);
    if (n0 + t < N && c < a.dc)
      *reinterpret_cast<u32x4_t*>(a.qa + ((long long)(n0 + t) * a.H + h) * a.dc + c) =
          *reinterpret_cast<const u32x4_t*>(lds + t * 272 + (tid & 15) * 16);
  }
}

// A tile is staged in two halves: 32 rows of the latent (64 chunks each, those
// past dc zeros), then 32 rows of r (8 chunks).  There is room for two tiles.
constexpr int DEC_HALF = 32, DEC_C = DEC_HALF * 1024, DEC_R = DEC_HALF * 128, DEC_BYTES = DEC_C + DEC_R;

// All but the newest half's loads have landed (ANY: 16 a wave, otherwise 9), in
// every wave.
template <bool ANY>
__device__ __forceinline__ void dec_sync() {
  if (ANY)
    asm volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else
    asm volatile("s_waitcnt vmcnt(9) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The request of tile t: the last b with first[b] <= t, by 64 probes at a time.
__device__ __forceinline__ int dec_request(const long long* first, int B, long long t, int lane) {
  int lo = 0, n = B;  // b is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) / 64, at = lo + lane * step;
    const int k = __popcll(__ballot(at < lo + n && first[at] <= t)) - 1;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// The waves of a row group (RG of them share a block, XN = 4 / RG waves each)
// split the tile twice: wave x forms the scores of 32 of the 64 keys (x % 2) and
// then adds up DC / XN columns of o~ over all 64, the weights passing through
// LDS in between.  So a lane holds all of its row's q~ and 1 / XN of o~, which
// fits the registers (a wave with all of o~, 256 of them, spilled; waves that
// each form all the scores spend half again as many products).  The rows of
// a group go by one reference point m for both halves of the keys: it is moved
// after a tile by the maxima that the waves have left, and a tile that
// passes it by more than 2^64 is formed again with the moved one (weights below
// 2^64 fit bf16 and fp32 as well as those below 1).  A piece's first tile is so
// formed twice, or with RG = 1 sets it between two more barriers, 1.5 us less
// (with RG = 2, whose registers are all taken, that spilled 14 and a batch of 128
// requests of 8000 tokens took 22 us longer).
//
// Loads: the second half of tile t + 1 goes out between the products that form
// the scores of tile t, the first half of tile t + 2 between the last products
// of tile t, whose own first half is then done with; so loads are under way all
// the time, and cost the one wave of a SIMD (an instruction in four cycles at
// best) no time of their own.  A wave's 8 rows of a half lie in one page where
// the page size is a multiple of 8, and come from one buffer that ends with the
// request's last row (later rows read as zeros).  Chunks past dc in a row's last
// 16 are r's and the next row's, which meet zeros of q~ and columns that are not
// kept.  ANY: other page sizes; each row is then looked up by itself (pages of
// 100 against 64, 131072 tokens, 128 heads: k_decode 81 against 57 us, with latents
// of 136 61 against 36).  A row takes 1024 bytes of LDS whatever dc is, so latents of
// 256 and fewer have the same visits at half the bytes and products (131072 tokens,
// 128 heads: 38 us of 256, 36 of 136).
template <int RG, int DC, bool ANY>
__global__ __launch_bounds__(256, 1) void k_decode(DecArgs a) {
  constexpr int XN = 4 / RG, CS = DC / 16, RS = 4, OT = DC / 32 / XN, ROWS = DEC_HALF / 4;
  constexpr int PL = RG == 1 ? 4096 : 0;  // the weights' second halves, after the first
  __shared__ __align__(1024) uint8_t lds[4 * DEC_BYTES + PL + RG * 4096 + RG * 256 + 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
  const int rg = wave % RG, x = wave / RG;
  uint8_t* pbuf = lds + 4 * DEC_BYTES + rg * 4096;                                    // the group's weights
  float* tops = reinterpret_cast<float*>(lds + 4 * DEC_BYTES + PL + RG * 4096) + rg * 64;  // and maxima
  int* far = reinterpret_cast<int*>(lds + 4 * DEC_BYTES + PL + RG * 4096 + RG * 256);      // a score passed m by 2^64
  // blocks of one worker on one XCD: they read the same rows
  const int bx = blockIdx.x & 7, by = blockIdx.x >> 3;
  const int worker = (by / a.row_blocks) * 8 + bx, rb = by % a.row_blocks;
  const long long total = a.first[a.B];
  const int workers = dec_workers(a, total);
  if (worker >= workers) return;
  const long long t1 = (worker + 1) * total / workers;
  const int R = a.S * a.H, row = (rb * RG + rg) * 32 + (lane & 31), width = a.dc + a.dr;
  const float sc = a.scale * LOG2E;
  const FragAt<64> fc(lane);
  const FragAt<8> fr(lane);
  // a lane's place in the eight rows of r of a wave
  const int rc = 8 * ((lane & 7) ^ swz<8>(8 * wave + (lane >> 3)));
  const uint32_t r_at = rc < a.dr ? ((lane >> 3) * width + a.dc + rc) * 2 : MLA_OOB;
  const uint32_t c_at = lane * 16 | (!ANY && 8 * (lane & ~15) >= a.dc ? MLA_OOB : 0);
  long long t = worker * total / workers;
  for (int b = dec_request(a.first, a.B, t, lane); t < t1; ++b) {
    const long long fb = a.first[b], next = a.first[b + 1];
    const int seq = a.seq_len[b];
    if (next <= t) continue;
    // kept in scalar registers, with all that follows from them
    const int ta = __builtin_amdgcn_readfirstlane((int)(t - fb)),
              tb = __builtin_amdgcn_readfirstlane((int)(min(next, t1) - fb)),
              len = __builtin_amdgcn_readfirstlane(dec_len(a, seq));
    const_i32* tab = (const_i32*)(a.table + (long long)__builtin_amdgcn_readfirstlane(b) * a.W);
    int bad = __builtin_amdgcn_readfirstlane((int)(seq > len));

    // The half to load next: its number, and page and place of the wave's first
    // row.  The page is read by a scalar load, one half before the rows (a vector
    // load would have to be waited for together with the rows in flight).
    int ahead = 2 * ta, page, off;
    auto split = [&](uint32_t j, uint32_t& p, uint32_t& o) {  // page and place in it
      p = __umulhi(j, a.inv_P), o = j - p * a.P;
      const uint32_t up = o >= (uint32_t)a.P;
      p += up, o -= up * a.P;
    };
    auto look_up = [&]() {
      uint32_t p, o;
      split(min(ahead * DEC_HALF + ROWS * wave, len - 1), p, o);
      page = tab[p];
      off = o;
    };
    auto address = [&](int page, int off) {
      const uint32_t in = (uint32_t)page < a.n_pages;
      bad |= in ^ 1;
      return a.cache + (long long)(in * (uint32_t)page * a.P + off) * width;  // a slot is below 2^31
    };
    // The loads of half `ahead` into its place, one at a time or all.
    uint32_t lo, hi, bytes;  // the buffer
    uint8_t *to_c, *to_r;
    uint32_t chunk;
    auto aim = [&]() {
      uint8_t* dst = lds + (ahead & 3) * DEC_BYTES;
      to_c = dst + ROWS * wave * 1024;
      to_r = dst + DEC_C + ROWS * wave * 128;
      const int first = ahead * DEC_HALF + ROWS * wave;
      chunk = c_at ^ ((wave & 1) * 32);  // row 8 of 16 and on: swz<64>(r + 8) = swz<64>(r) ^ 2
      asm volatile("" : "+v"(chunk));    // the offsets are not to be kept in registers
      if (!ANY) {
        const int end = min(len, tb * DEC_TILE);  // nothing past the piece
        const unsigned long long p = reinterpret_cast<unsigned long long>(address(page, off));
        lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
        bytes = __builtin_amdgcn_readfirstlane(max(0, min(ROWS, end - first)) * width * 2);
      } else {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {  // rows past the end: the last
          uint32_t p, o;
          split(min(first + r, len - 1), p, o);
          const uint16_t* at = address(tab[p], o);
          mla_dma16(mla_rsrc(at, a.dc * 2), to_c + r * 1024, chunk ^ (swz<64>(r) * 16));
          if ((lane >> 3) == r)
            mla_dma16(mla_rsrc(at + a.dc, a.dr * 2), to_r, ((lane & 7) ^ swz<8>(8 * wave + r)) * 16);
        }
      }
      ++ahead;
    };
    auto load = [&](int j) {
      if (ANY) return;
      const __amdgpu_buffer_rsrc_t rs = mla_rsrc(reinterpret_cast<const void*>((unsigned long long)hi << 32 | lo), bytes);
      if (j < ROWS)
        mla_dma16(rs, to_c + j * 1024, (chunk ^ (swz<64>(j) * 16)) + j * width * 2);
      else if (j == ROWS)
        mla_dma16(rs, to_r, r_at);
    };
    look_up();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      aim();
#pragma unroll
      for (int j = 0; j <= ROWS; ++j) load(j);
      look_up();
    }

    // queries, one row to a column
    bf16x8_t q[CS + RS];
    const long long qrow = (long long)b * R + min(row, R - 1);
#pragma unroll
    for (int k = 0; k < CS; ++k) q[k] = load8(a.qa + qrow * a.dc, 16 * k + 8 * half, row < R && 16 * k + 8 * half < a.dc);
#pragma unroll
    for (int k = 0; k < RS; ++k)
      q[CS + k] = load8(a.q + qrow * (a.dn + a.dr) + a.dn, 16 * k + 8 * half, row < R && 16 * k + 8 * half < a.dr);
    const int vis = len - (a.S - 1 - min(row, R - 1) / a.H), all = len - (a.S - 1);

    float m = -INFINITY, l = 0.f;
    f32x16_t o[OT];
#pragma unroll
    for (int d = 0; d < OT; ++d) o[d] = zero16();
    // the queries have landed: with their loads open the compiler would wait for
    // all loads in each turn
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    int i = ta;
    while (i < tb) {
      // The sums stay in place through the inner loop, which is left when the
      // reference point moves.
      float top;
      bool again;
      do {
        const int h0 = 2 * (i & 1), key0 = i * DEC_TILE + (x & 1) * DEC_HALF;
        const uint8_t *c0 = lds + h0 * DEC_BYTES, *mine = c0 + (x & 1) * DEC_BYTES;
        dec_sync<ANY>();
        aim();
        auto ac = fc.fresh();
        const auto ar = fr.fresh();
        f32x16_t s = zero16();
        auto key = [&](int k) { return k < CS ? frag_row(mine, ac, 0, k) : frag_row(mine + DEC_C, ar, 0, k - CS); };
        Ahead<CS + RS, 6> qk;
        qk.start(key);
        qk.run(key, [&](int k, bf16x8_t f) {
          s = mma(f, q[k], s);
          if (k % 2 == 1) load(k / 2);
        });
        look_up();
        if (key0 + DEC_HALF > all) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (key0 + 8 * (r >> 2) + 4 * half + (r & 3) >= vis) s[r] = -INFINITY;
        }
        ac.tr ^= ((x * OT) & 3) << 6;
        auto col = [&](int k) {
          return frag_tr(c0 + (k / OT >> 1) * DEC_BYTES + ((x * OT) >> 2) * 256, ac, 16 * (k / OT & 1), k % OT);
        };
        Ahead<4 * OT, 4> pv;
        pv.start(col);
        top = s[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
        top = max_halves(top) * sc;
        if (RG == 1 && i == ta && m == -INFINITY) {
          if (x < 2 && half == 0) lds_put(tops + (x & 1) * 32 + lane, top);
          mla_sync_lds();
          m = fmaxf(lds_get<float>(tops + (lane & 31)), lds_get<float>(tops + 32 + (lane & 31)));
          mla_sync_lds();
        }
        const float ms = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -ms));
          sum += s[r];
        }
        if (x < 2) {
#pragma unroll
          for (int k = 0; k < 2; ++k) lds_put(pbuf + x * 2048 + k * 1024 + lane * 16, pack8(s, 8 * k));
          if (RG == 1) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] -= bf16_to_f32(f32_to_bf16(s[r]));
#pragma unroll
            for (int k = 0; k < 2; ++k) lds_put(pbuf + PL + x * 2048 + k * 1024 + lane * 16, pack8(s, 8 * k));
          }
          if (half == 0) lds_put(tops + (x & 1) * 32 + lane, top);
        }
        const int passed = wave_any(top > m + 64.f);
        if (lane == 0) lds_put(far + wave, passed);
        mla_sync_lds();
        const int4 f = lds_get<int4>(far);
        bf16x8_t p[4], pl[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = lds_get<bf16x8_t>(pbuf + k * 1024 + lane * 16);
        if (RG == 1) {
#pragma unroll
          for (int k = 0; k < 4; ++k) pl[k] = lds_get<bf16x8_t>(pbuf + PL + k * 1024 + lane * 16);
        }
        top = fmaxf(lds_get<float>(tops + (lane & 31)), lds_get<float>(tops + 32 + (lane & 31)));
        again = __builtin_amdgcn_readfirstlane(f.x | f.y | f.z | f.w) != 0;
        if (again) break;
        l += sum;
        auto use = [&](int k, bf16x8_t f) {
          o[k % OT] = mma(f, p[k / OT], o[k % OT]);
          if (RG == 1) o[k % OT] = mma(f, pl[k / OT], o[k % OT]);
        };
        pv.template run<0, 2 * OT>(col, use);
        mla_sync_lds();  // every wave is done with the first half
        aim();
        pv.template run<2 * OT, 4 * OT>(col, [&](int k, bf16x8_t f) {
          use(k, f);
          load(k - 2 * OT);
        });
#pragma unroll
        for (int j = 2 * OT; j <= ROWS; ++j) load(j);
        look_up();
        ++i;
      } while (i < tb && !wave_any(top > m + 8.f));
      rescale(m, l, o, top);
      if (again) {  // once more from dec_sync() on, the loads too
        --ahead;
        look_up();
      }
    }
    l = sum_halves(l);
    mla_sync();  // the loads past the end have landed, and every wave is done with the tiles
    if (x < 2 && half == 0) tops[(x & 1) * 32 + lane] = l;
    if (lane == 0) far[wave] = bad;
    mla_sync_lds();
    l = lds_get<float>(tops + (lane & 31)) + lds_get<float>(tops + 32 + (lane & 31));
    const int4 f = lds_get<int4>(far);
    if (f.x | f.y | f.z | f.w) l = __builtin_nanf("");
    if (row < R) {
      const long long piece = ((long long)worker + b) * R + row;
#pragma unroll
      for (int d = 0; d < OT; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int col = 32 * (x * OT + d) + 2 * r + 4 * half;
          if (col < a.dc)
            store4(a.o, piece * a.dc + col, false, o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]);
        }
      if (half == 0 && x == 0) a.ml[2 * piece] = m, a.ml[2 * piece + 1] = l;
    }
    t = fb + tb;
  }
}

// A share of one row's pieces in the order of their workers: w0, w0 + step, ..
// up to w1.  Lane l takes columns 8 l .. + 7.  The maxima and sums of 64 pieces
// are read at once, a piece to a lane, and the first eight pieces with them, so
// that those loads depend on nothing.  (W^V read before the join too, half of it
// by each of eight waves, took another 1.5 us of 85 from one long request and
// nothing from others: not worth a second form.)
struct Joined {
  float m, l, v[8];
};
__device__ __forceinline__ Joined dec_join(const DecArgs& a, int b, int row, int w0, int w1, int step, int lane) {
  const int R = a.S * a.H;
  const bool live = 8 * lane < a.dc;
  Joined j{-INFINITY, 0.f, {}};
  for (; w0 <= w1; w0 += 64 * step) {
    const int n = min(64, (w1 - w0) / step + 1);
    const long long piece0 = ((long long)w0 + b) * R + row, stride = (long long)step * R;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = *reinterpret_cast<const float2*>(a.ml + 2 * (piece0 + lane * stride));
    const float* p = a.o + piece0 * a.dc + (live ? 8 * lane : 0);
    float4 x[8][2];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < n) {
          const float4* q = reinterpret_cast<const float4*>(p + (k0 + k) * stride * a.dc);
          x[k][0] = q[0], x[k][1] = q[1];
        }
    };
    load(0);
    const float top = fmaxf(j.m, wave_max_f32(ml.x)), ms = top == -INFINITY ? 0.f : top;
    const float f = __builtin_amdgcn_exp2f(j.m - ms), w = __builtin_amdgcn_exp2f(ml.x - ms);
    float l = lane < n ? ml.y * w : 0.f;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off, 64);
    j.m = top;
    j.l = j.l * f + l;
#pragma unroll
    for (int i = 0; i < 8; ++i) j.v[i] *= f;
    for (int k0 = 0; k0 < n; k0 += 8) {
      if (k0 > 0) load(k0);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < n) {
          const float g = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), k0 + k));
          const float t[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) j.v[i] = fmaf(t[i], g, j.v[i]);
        }
    }
  }
  return j;
}

// o = W^V o~ for a head and up to 32 tokens.  The rows' pieces are joined first:
// a row to a wave, or where the tokens are fewer than the eight waves, a row's
// pieces dealt to several.  o~ goes into LDS as two bf16 halves (chunk c of token t at
// c ^ swz(t)), and each of four waves multiplies 32 rows of W^V with both.
template <int DC>
__global__ __launch_bounds__(512, 4) void k_out(DecArgs a, void* out, bool out_bf16, int tokens) {
  __shared__ __align__(16) uint8_t lds[2 * 32 * DC * 2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
  const int N = a.B * a.S, R = a.S * a.H, h = blockIdx.x % a.H, n0 = blockIdx.x / a.H * tokens,
            live = min(tokens, N - n0);
  const int v = 32 * (wave & 3) + (lane & 31);
  const uint16_t* wp = a.w + ((long long)h * (a.dn + a.dv) + a.dn + min(v, a.dv - 1)) * a.dc;

  const long long total = a.first[a.B];
  const int G = dec_workers(a, total);
  auto join = [&](int t, int slice, int slices) {
    const int n = n0 + t, b = n / a.S, row = (n - b * a.S) * a.H + h;
    const long long f0 = a.first[b], f1 = a.first[b + 1];
    if (f1 == f0) return Joined{-INFINITY, 0.f, {}};
    return dec_join(a, b, row, dec_worker(f0, total, G) + slice, dec_worker(f1 - 1, total, G), slices, lane);
  };
  auto keep = [&](int t, const Joined& j) {
    const float inv = j.l == 0.f ? 0.f : 1.0f / j.l;
    u32x4_t hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = j.v[2 * i] * inv, y = j.v[2 * i + 1] * inv;
      const uint32_t p = pack_bf16x2(x, y);
      hi[i] = p;
      lo[i] = pack_bf16x2(x - __uint_as_float(p << 16), y - __uint_as_float(p & 0xFFFF0000u));
    }
    if (8 * lane < DC) {
      const int at = t * DC * 2 + ((lane ^ swz<16>(t)) << 4);
      const u32x4_t z = {0, 0, 0, 0};
      *reinterpret_cast<u32x4_t*>(lds + at) = 8 * lane < a.dc ? hi : z;
      *reinterpret_cast<u32x4_t*>(lds + 32 * DC * 2 + at) = 8 * lane < a.dc ? lo : z;
    }
  };
  if (live >= 8) {
    for (int t = wave; t < live; t += 8) keep(t, join(t, 0, 1));
  } else {
    const int slices = 8 / live, t = wave % live, slice = wave / live;
    float* part = reinterpret_cast<float*>(lds);  // of each wave: 8 columns a lane, then m and l
    Joined j = join(t, min(slice, slices - 1), slices);
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave * 520 + 64 * i + lane] = j.v[i];
    if (lane == 0) part[wave * 520 + 512] = j.m, part[wave * 520 + 513] = j.l;
    __syncthreads();
    if (wave < live) {  // the row's slices in their order
      for (int s = 1; s < slices; ++s) {
        const float* p = part + (wave + s * live) * 520;
        const float mn = fmaxf(j.m, p[512]), ms = mn == -INFINITY ? 0.f : mn;
        const float f = __builtin_amdgcn_exp2f(j.m - ms), g = __builtin_amdgcn_exp2f(p[512] - ms);
        j.m = mn;
        j.l = j.l * f + p[513] * g;
#pragma unroll
        for (int i = 0; i < 8; ++i) j.v[i] = j.v[i] * f + p[64 * i + lane] * g;
      }
    }
    __syncthreads();
    if (wave < live) keep(wave, j);
  }
  __syncthreads();
  if (wave >= 4) return;
  f32x16_t o = zero16();
#pragma unroll
  for (int k0 = 0; k0 < DC / 16; k0 += 16) {
    bf16x8_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = load8(wp, 16 * (k0 + k) + 8 * half, 16 * (k0 + k) + 8 * half < a.dc);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int t = lane & 31, at = t * DC * 2 + (((2 * (k0 + k) + half) ^ swz<16>(t)) << 4);
      o = mma(w[k], *reinterpret_cast<const bf16x8_t*>(lds + at), o);
      o = mma(w[k], *reinterpret_cast<const bf16x8_t*>(lds + 32 * DC * 2 + at), o);
    }
  }
  const int n = n0 + (lane & 31);
  if ((lane & 31) >= live) return;
  store_tile(out, ((long long)n * a.H + h) * a.dv + 32 * wave, out_bf16, o, 1.f, half, a.dv - 32 * wave);
}

// How the work is divided: row groups of 32 a block, and runs of tiles, one
// block a CU in all (the staged tiles take 144 KB of LDS).
struct DecPlan {
  int rg, row_blocks, workers;
};
DecPlan dec_plan(long long B, long long S, long long H, long long max_len) {
  const long long R = S * H, tiles = B * ceil_div(max_len > 0 ? max_len : 1, DEC_TILE);
  // 64 rows a block read the cache half as often as 32 (131072 tokens, 128 heads: 74
  // us a call for 96); where the tiles leave CUs idle, 32 (4 requests of 300 tokens:
  // 30 us for 34)
  int rg = R > 32 ? 2 : 1;
  if (rg > 1 && tiles * ceil_div(R, 32 * rg) < DEC_CUS) rg = 1;
  const long long rb = ceil_div(R, 32 * rg);
  long long workers = DEC_CUS / rb;
  if (workers > tiles) workers = tiles;
  return {rg, (int)rb, (int)(workers < 1 ? 1 : workers)};
}

struct DecSpace {
  size_t qa, o, ml, first, bytes;
};
DecSpace dec_space(const DecPlan& p, long long B, long long S, long long H, long long dc) {
  auto up = [](long long n) { return (size_t)ceil_div(n, 256) * 256; };
  const long long N = B * S, pieces = (p.workers + B) * S * H;
  DecSpace s;
  s.qa = 0;
  s.o = s.qa + up(N * H * dc * 2);
  s.ml = s.o + up(pieces * dc * 4);
  s.first = s.ml + up(pieces * 8);
  s.bytes = s.first + up((B + 1) * 8);
  return s;
}

bool dec_sizes_ok(int B, int S, int H, int dn, int dr, int dv, int dc, long long max_len) {
  return B >= 1 && B <= DEC_MAX_B && S >= 1 && S <= 64 && H >= 1 && H <= 1024 &&
         (long long)B * S * H <= DEC_MAX_ROWS && mla_dims_ok(dn, dr, dv) &&
         mla_dc_ok(dc) && max_len >= 0;
}

}  // namespace

size_t decode_workspace_bytes(int B, int S, int H, int dn, int dr, int dv, int dc, long long max_len) {
  if (!dec_sizes_ok(B, S, H, dn, dr, dv, dc, max_len)) return 0;
  return dec_space(dec_plan(B, S, H, max_len), B, S, H, dc).bytes;
}

moe_status decode(const void* q, const void* w, const void* cache, long long n_pages, int page_size,
                  const int32_t* table, int W, const int32_t* seq_len, int B, int S, int H, int dn, int dr, int dv,
                  int dc, long long max_len, float scale, void* out, moe_dtype out_t, void* ws, size_t ws_bytes,
                  void* stream) {
  MOE_REQUIRE(B >= 0 && S >= 1 && H >= 1 && W >= 1 && page_size >= 1 && n_pages >= 0 && max_len >= 0, MOE_EINVAL,
              "need B, n_pages, max_len >= 0 and S, H, W, page_size >= 1");
  MOE_REQUIRE(dn >= 8 && dr >= 8 && dv >= 8 && dc >= 8 && dn % 8 == 0 && dr % 8 == 0 && dv % 8 == 0 && dc % 8 == 0,
              MOE_EINVAL, "dn, dr, dv and dc must be positive multiples of 8");
  MOE_REQUIRE(mla_dims_ok(dn, dr, dv) && mla_dc_ok(dc), MOE_EUNSUPPORTED,
              "dn or dv above 128, dr above 64 or dc above 512");
  MOE_REQUIRE(B <= DEC_MAX_B && S <= 64 && H <= 1024, MOE_EUNSUPPORTED,
              "more requests than MLA_MAX_REQUESTS, S above 64 or H above 1024");
  MOE_REQUIRE(n_pages * page_size < (1LL << 31), MOE_EUNSUPPORTED, "2^31 slots or more");
  MOE_REQUIRE((long long)B * S * H <= DEC_MAX_ROWS, MOE_EUNSUPPORTED, "more than 2^26 queries");
  MOE_REQUIRE(mla_scale_ok(scale), MOE_EINVAL, "scale must be positive and at most 2^127");
  MOE_REQUIRE(out_t == MOE_F32 || out_t == MOE_BF16, MOE_EINVAL, "out_t must be MOE_F32 or MOE_BF16");
  if (B == 0) return MOE_OK;
  MOE_REQUIRE(q && w && table && seq_len && out && cache && n_pages > 0, MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(w) && aligned16(cache) && aligned16(out) && aligned16(ws), MOE_EINVAL,
              "q, w_kv, cache, out and ws must be 16-byte aligned");
  const DecPlan p = dec_plan(B, S, H, max_len);
  const DecSpace sp = dec_space(p, B, S, H, dc);
  MOE_REQUIRE(ws && ws_bytes >= sp.bytes, MOE_EWORKSPACE, "workspace smaller than mla_decode_workspace_bytes");
  char* base = static_cast<char*>(ws);
  const DecArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(w), static_cast<const uint16_t*>(cache),
                  table, seq_len, B, S, H, dn, dr, dv, dc, W, page_size, (uint32_t)n_pages, scale, p.workers, p.row_blocks,
                  page_size == 1 ? 0xFFFFFFFFu : (uint32_t)((1ULL << 32) / page_size),
                  reinterpret_cast<uint16_t*>(base + sp.qa), reinterpret_cast<float*>(base + sp.o),
                  reinterpret_cast<float*>(base + sp.ml), reinterpret_cast<long long*>(base + sp.first)};
  hipStream_t st = as_stream(stream);
  const long long N = (long long)B * S;
  hipLaunchKernelGGL(k_absorb, dim3((unsigned)(ceil_div(dc, 128) * H * ceil_div(N, 32))), dim3(256), 0, st, a);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(ceil_div(p.workers, 8) * 8 * p.row_blocks)), dim3(256), 0, st, a);
  };
  // latents up to 256 by kernels of half the registers and products: 16384 tokens of
  // 256, 128 heads, 31 us a call for 36, 131072 52 for 63
  auto pick = [&](auto any) {
    constexpr bool ANY = decltype(any)::value;
    if (dc <= 256) {
      if (p.rg == 2) go(k_decode<2, 256, ANY>); else go(k_decode<1, 256, ANY>);
    } else {
      if (p.rg == 2) go(k_decode<2, 512, ANY>); else go(k_decode<1, 512, ANY>);
    }
  };
  if (page_size % 8 == 0)
    pick(std::false_type{});
  else
    pick(std::true_type{});
  // Fewer tokens a block where there would be less than a block a CU: the pieces'
  // loads bound it.  Against 32 everywhere, whole calls: 16 requests of 1000 tokens,
  // 32 heads, 34.7 for 39.7 us, 31 of 6000 with 4 tokens each, 8 heads, 64 for 73;
  // up to two blocks a CU the more reads of W^V cost as much again: 100 requests of
  // 500 tokens, 64 heads, 73 for 64 us.
  int tokens = 32;
  while (tokens > 4 && H * ceil_div(N, tokens) < DEC_CUS) tokens /= 2;
  hipLaunchKernelGGL(dc <= 256 ? k_out<256> : k_out<512>, dim3((unsigned)(H * ceil_div(N, tokens))), dim3(512), 0, st,
                     a, out, out_t == MOE_BF16, tokens);
  return launch_status("mla_decode");
}

}  // namespace moe
