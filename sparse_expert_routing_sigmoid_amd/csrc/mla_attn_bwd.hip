// Gradient of the expanded latent attention (mla_attn.hip), given dO:
//   P_ij = exp(s_ij - lse_i),  D_i = sum_d dO_id o_id
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dr_j = sum over the heads of dK's
//   rotary columns
// Two kernels that each form S and dP, so that every gradient is summed by one
// wave in a fixed order (no atomics: results are bitwise reproducible): k_attn_dq
// walks the keys of 128 queries as the forward does and leaves D and lse (in
// powers of two), k_attn_dkv walks the queries of 128 keys.  That is seven
// products of 2 dqk or 2 dv flops a visible pair and head, 2 (4 dqk + 3 dv), where
// five, 2 (3 dqk + 2 dv), would do if dQ were added up across blocks: by atomics,
// whose order changes the sums' bits, or from dS kept in memory, 2 GB of bf16 at
// 4096 tokens and 128 heads.  (A head's causal half of that is 16 MB, so a few heads
// at a time would stay in the last-level cache: not measured.)  P and dS are rounded to bf16 for their products, to
// the nearest (2^-8 of a term at most, of either sign; the sums stay fp32).
// k_attn_dr adds the heads' parts of dr, which k_attn_dkv leaves in fp32.
#include <type_traits>

#include "mla.h"
#include "mla_attn.h"

namespace moe {

namespace {

// As k_attn_fwd: 32 queries to a wave, tiles of 64 keys in two stages, two
// blocks a CU.  4096 tokens, 128 heads, causal: 1050 us, 1047 TFLOP/s of its three
// products, MFMA busy 57 % of the cycles at 1.8 GHz.
template <int DN, int DR, int DV>
__global__ __launch_bounds__(256, 2) void k_attn_dq(AttnArgs a, const uint16_t* __restrict__ dout, const void* out,
                                                    bool out_bf16, const float* __restrict__ lse, void* dq, bool g_bf16,
                                                    float* __restrict__ stat) {
  using T = KeyTile<DN, DR, DV>;
  constexpr int KS = DN / 16, RS = DR / 16, VS = DV / 16, NT = DN / 32, RT = DR / 32;
  __shared__ __align__(16) uint8_t lds[2 * T::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  int h;
  const AttnTile seq = attn_find(a, h, lds);
  if (seq.row0 < 0) return;

  const int i = seq.row0 + wave * 32 + (lane & 31);
  const bool live = i < seq.lq;
  const long long row = (seq.q0 + (live ? i : 0)) * a.H + h;
  const uint16_t *qp = a.q + row * (a.dn + a.dr), *dp_ = dout + row * a.dv;
  bf16x8_t q[KS + RS], g[VS];
#pragma unroll
  for (int s = 0; s < KS; ++s) q[s] = load8(qp, 16 * s + 8 * half, live && 16 * s + 8 * half < a.dn);
#pragma unroll
  for (int s = 0; s < RS; ++s) q[KS + s] = load8(qp + a.dn, 16 * s + 8 * half, live && 16 * s + 8 * half < a.dr);
  float D = 0.f;
#pragma unroll
  for (int s = 0; s < VS; ++s) {
    const int c = 16 * s + 8 * half;
    g[s] = load8(dp_, c, live && c < a.dv);
    if (live && c < a.dv) {
      if (out_bf16) {
        const bf16x8_t o = load8(static_cast<const uint16_t*>(out) + row * a.dv, c, true);
#pragma unroll
        for (int e = 0; e < 8; ++e) D = fmaf((float)g[s][e], (float)o[e], D);
      } else {
        const float* o = static_cast<const float*>(out) + row * a.dv + c;
#pragma unroll
        for (int e = 0; e < 8; ++e) D = fmaf((float)g[s][e], o[e], D);
      }
    }
  }
  D = sum_halves(D);
  const float sc = a.scale * LOG2E, ls = live ? lse[row] * LOG2E : 0.f;
  if (live && half == 0) *reinterpret_cast<float2*>(stat + 2 * row) = make_float2(ls, D);

  const int vis = !live ? 0 : a.causal ? min(seq.lk, i + seq.lk - seq.lq + 1) : seq.lk;
  const int last = min(seq.lq, seq.row0 + 128) - 1;
  const int end = a.causal ? min(seq.lk, last + seq.lk - seq.lq + 1) : seq.lk;
  const int tiles = end > 0 ? (end + 63) / 64 : 0;
  const int wrow = seq.row0 + wave * 32, wlast = min(seq.lq, wrow + 32) - 1;
  const int all = wrow >= seq.lq ? 0 : a.causal ? min(seq.lk, wrow + seq.lk - seq.lq + 1) : seq.lk;
  const int none = wrow >= seq.lq ? 0 : a.causal ? min(seq.lk, wlast + seq.lk - seq.lq + 1) : seq.lk;

  T tile;
  tile.init(a, h, seq.k0, max(end, 0), lane, wave);
  const FragAt<T::CN> fn(lane);
  const FragAt<T::CR> fr(lane);
  const FragAt<T::CV> fv(lane);
  f32x16_t ak[NT + RT];
#pragma unroll
  for (int d = 0; d < NT + RT; ++d) ak[d] = zero16();

  tile.load_all(lds, 0);
  auto turn = [&](int t, auto masked) {
    mla_sync();
    tile.aim(lds + ((t + 1) & 1) * T::BYTES, t + 1);
    const uint8_t *kn = lds + (t & 1) * T::BYTES, *kr = kn + T::KN, *v = kr + T::KR;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const auto an = fn.fresh();
      const auto ar = fr.fresh();
      const auto av = fv.fresh();
      f32x16_t s = zero16(), p = zero16();
      constexpr int NF = KS + RS + VS, NB = 2 * (NT + RT);
      auto front = [&](int k) {  // S, then dP
        return k < KS        ? frag_row(kn, an, 32 * u, k)
               : k < KS + RS ? frag_row(kr, ar, 32 * u, k - KS)
                             : frag_row(v, av, 32 * u, k - KS - RS);
      };
      Ahead<NF, 3> f;
      f.start(front);
      f.run(front, [&](int k, bf16x8_t x) {
        if (k < KS + RS)
          s = mma(x, q[k], s);
        else
          p = mma(x, g[k - KS - RS], p);
        if (u == 0) tile.load(k);
      });
      auto tail = [&](int k) {
        const int kk = k / (NT + RT), d = k % (NT + RT);
        return d < NT ? frag_tr(kn, an, 32 * u + 16 * kk, d) : frag_tr(kr, ar, 32 * u + 16 * kk, d - NT);
      };
      Ahead<NB, 3> b;
      b.start(tail);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -ls)) * (p[r] - D);
        if (decltype(masked)::value)
          if (64 * t + 32 * u + 8 * (r >> 2) + 4 * half + (r & 3) >= vis) s[r] = 0.f;
      }
      const bf16x8_t ds[2] = {pack8(s, 0), pack8(s, 8)};
      b.run(tail, [&](int k, bf16x8_t x) { ak[k % (NT + RT)] = mma(x, ds[k / (NT + RT)], ak[k % (NT + RT)]); });
    }
  };
  const int whole = min(tiles, max(0, all / 64)), some = min(tiles, max(0, none + 63) / 64);
  int t = 0;
  for (; t < whole; ++t) turn(t, std::false_type{});
  for (; t < some; ++t) turn(t, std::true_type{});
  for (; t < tiles; ++t) {
    mla_sync();
    tile.load_all(lds + ((t + 1) & 1) * T::BYTES, t + 1);
  }
  __builtin_amdgcn_s_waitcnt(WAIT_VM0);  // no load into LDS outlives the block
  if (!live) return;
#pragma unroll
  for (int d = 0; d < NT + RT; ++d) {
    const int c = 32 * (d < NT ? d : d - NT);
    store_tile(dq, row * (a.dn + a.dr) + (d < NT ? 0 : a.dn) + c, g_bf16, ak[d], a.scale, half,
               (d < NT ? a.dn : a.dr) - c);
  }
}

// The two waves of a pair share 32 keys and split the work on them: the first
// forms S and P and adds up dV, the second forms dP and dS and adds up dK, taking
// P from LDS one step of 32 queries later.  Each has as many products (20 a
// step), and with half of the sums two waves fit a SIMD, one of each kind: one
// issues while the other waits.  Query tiles are staged four deep: the second
// wave is one behind, and two are in flight.
// 4096 tokens, 128 heads, causal: 1555 us, 885 TFLOP/s of these products; the MFMA
// pipe is busy 46 % of the cycles at 1.9 GHz.  Measured against it: one wave of 32
// keys and all four products a SIMD, with every fragment read ahead and the
// arithmetic spread between the products, 1581 us; pairs on 64 keys, one wave a
// SIMD, 1667; dK added up a step later, so that one kind's products run beside
// the other's arithmetic, and a fifth stage for it, 0.5 % less: not kept; two, six
// or seven fragments read ahead instead of four, 1 to 2 % more.
template <int DN, int DR, int DV>
__global__ __launch_bounds__(512, 1) void k_attn_dkv(AttnArgs a, const uint16_t* __restrict__ dout,
                                                     const float* __restrict__ stat, void* dkv, bool g_bf16,
                                                     float* __restrict__ dr_part) {
  using T = QueryTile<DN, DR, DV>;
  constexpr int KS = DN / 16, RS = DR / 16, KF = KS + RS, VS = DV / 16, NT = DN / 32, NK = NT + DR / 32, VT = DV / 32;
  constexpr int PB = 16 * 64 * 4;  // P of one pair and step
  __shared__ __align__(16) uint8_t lds[4 * T::BYTES + 2 * 4 * PB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int pair = wave & 3;
  int h;
  const AttnTile seq = attn_find<8>(a, h, lds);
  if (seq.row0 < 0) return;

  // this pair's keys, one to a column
  const int key = seq.row0 + 32 * pair + (lane & 31);
  const bool live = key < seq.lk;
  const long long row = (seq.k0 + min(key, seq.lk - 1)) * a.H + h;
  const int back = a.causal ? seq.lk - seq.lq : seq.lk;  // query i sees keys j <= i + back
  const int begin = a.causal ? max(0, seq.row0 - back) / 32 : 0, steps = (seq.lq + 31) / 32;
  // from this tile on every query sees every key of the pair
  const int whole = a.causal ? max(0, min(seq.row0 + 32 * pair + 31, seq.lk - 1) - back + 31) / 32 : 0;
  const int first = a.causal ? key - back : 0;  // the first query that sees this lane's key
  uint8_t* pbuf = lds + 4 * T::BYTES + pair * PB + lane * 16;  // + 4 PB for odd steps

  T tile;
  tile.init(a, dout, stat, h, seq.q0, seq.lq, lane, wave);
  const FragAt<T::CN> fn(lane);
  const FragAt<T::CR> fr(lane);
  const FragAt<T::CV> fv(lane);
  const float sc = a.scale * LOG2E;
  if (begin < steps) {
    tile.load_all(lds + (begin & 3) * T::BYTES, begin);
    tile.load_all(lds + ((begin + 1) & 3) * T::BYTES, begin + 1);
  }
  // tile n has landed and tile n - 2 is done with
  auto sync = [&](int n) {
    static_assert(T::LOADS == 4, "the count below");
    asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    tile.aim(lds + ((n + 2) & 3) * T::BYTES, n + 2);
  };

  if (wave < 4) {
    bf16x8_t kf[KF];
    const uint16_t *kp = a.kv + row * (a.dn + a.dv), *rp = a.k_rope + (seq.k0 + min(key, seq.lk - 1)) * a.ldr;
#pragma unroll
    for (int s = 0; s < KS; ++s) kf[s] = load8(kp, 16 * s + 8 * half, live && 16 * s + 8 * half < a.dn);
#pragma unroll
    for (int s = 0; s < RS; ++s) kf[KS + s] = load8(rp, 16 * s + 8 * half, live && 16 * s + 8 * half < a.dr);
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    f32x16_t dv[VT];
#pragma unroll
    for (int d = 0; d < VT; ++d) dv[d] = zero16();
    auto turn = [&](int n, auto masked) {
      sync(n);
      const uint8_t *qn = lds + (n & 3) * T::BYTES, *qr = qn + T::QN, *go = qr + T::QR, *st = go + T::DO;
      const auto an = fn.fresh();
      const auto ar = fr.fresh();
      const auto ao = fv.fresh();
      auto line = [&](int k) { return k < KS ? frag_row(qn, an, 0, k) : frag_row(qr, ar, 0, k - KS); };
      auto col = [&](int k) { return frag_tr(go, ao, 16 * (k / VT), k % VT); };
      f32x16_t s = zero16();
      bf16x8_t w[2];
      float4 ls;
      auto weight = [&](int r) {
        if (r % 4 == 0) ls = lds_get<float4>(st + (2 * r + 4 * half) * 4);
        const float e = r % 4 == 0 ? ls.x : r % 4 == 1 ? ls.y : r % 4 == 2 ? ls.z : ls.w;
        s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -e));
        if (decltype(masked)::value)
          if (32 * n + 8 * (r >> 2) + 4 * half + (r & 3) < first) s[r] = 0.f;
        if (r % 4 == 3)
          lds_put(pbuf + (n & 1) * 4 * PB + (r / 4) * 1024, make_float4(s[r - 3], s[r - 2], s[r - 1], s[r]));
        if (r % 8 == 7) w[r / 8] = pack8(s, r - 7);
      };
      Ahead<KF, 4> f;
      f.start(line);
      f.run(line, [&](int k, bf16x8_t x) {
        s = mma(x, kf[k], s);
        tile.load(k);
      });
      Ahead<2 * VT, 4> g;
      g.start(col);
#pragma unroll
      for (int r = 0; r < 8; ++r) weight(r);
      g.run(col, [&](int k, bf16x8_t x) {
        dv[k % VT] = mma(x, w[k / VT], dv[k % VT]);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r * VT / 8 == k) weight(8 + r);
      });
    };
    int n = begin;
    const int some = min(steps, max(begin, whole));
    for (; n < some; ++n) turn(n, std::true_type{});
    for (; n < steps; ++n) turn(n, std::false_type{});
    if (begin < steps) sync(n);  // the other wave's last step
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);  // no load into LDS outlives the block
    if (!live) return;
#pragma unroll
    for (int d = 0; d < VT; ++d)
      store_tile(dkv, row * (a.dn + a.dv) + a.dn + 32 * d, g_bf16, dv[d], 1.f, half, a.dv - 32 * d);
  } else {
    bf16x8_t vf[VS];
    const uint16_t* vp = a.kv + row * (a.dn + a.dv) + a.dn;
#pragma unroll
    for (int s = 0; s < VS; ++s) vf[s] = load8(vp, 16 * s + 8 * half, live && 16 * s + 8 * half < a.dv);
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    f32x16_t dk[NK];
#pragma unroll
    for (int d = 0; d < NK; ++d) dk[d] = zero16();
    auto turn = [&](int n, auto masked) {  // of tile n - 1
      sync(n);
      const uint8_t *qn = lds + ((n - 1) & 3) * T::BYTES, *qr = qn + T::QN, *go = qr + T::QR, *st = go + T::DO + 128;
      const auto an = fn.fresh();
      const auto ar = fr.fresh();
      const auto ao = fv.fresh();
      auto line = [&](int k) { return frag_row(go, ao, 0, k); };
      auto col = [&](int k) {
        const int kk = k / NK, d = k % NK;
        return d < NT ? frag_tr(qn, an, 16 * kk, d) : frag_tr(qr, ar, 16 * kk, d - NT);
      };
      f32x16_t p = zero16();
      bf16x8_t ds[2];
      float4 dd, w;
      auto grad = [&](int r) {
        if (r % 4 == 0) {
          dd = lds_get<float4>(st + (2 * r + 4 * half) * 4);
          w = lds_get<float4>(pbuf + ((n - 1) & 1) * 4 * PB + (r / 4) * 1024);
        }
        const float e = r % 4 == 0 ? dd.x : r % 4 == 1 ? dd.y : r % 4 == 2 ? dd.z : dd.w;
        const float f = r % 4 == 0 ? w.x : r % 4 == 1 ? w.y : r % 4 == 2 ? w.z : w.w;
        p[r] = f * (p[r] - e);
        if (decltype(masked)::value)
          if (32 * (n - 1) + 8 * (r >> 2) + 4 * half + (r & 3) < first) p[r] = 0.f;
        if (r % 8 == 7) ds[r / 8] = pack8(p, r - 7);
      };
      Ahead<VS, 4> f;
      f.start(line);
      f.run(line, [&](int k, bf16x8_t x) {
        p = mma(x, vf[k], p);
        tile.load(k);
      });
      Ahead<2 * NK, 4> g;
      g.start(col);
#pragma unroll
      for (int r = 0; r < 8; ++r) grad(r);
      g.run(col, [&](int k, bf16x8_t x) {
        dk[k % NK] = mma(x, ds[k / NK], dk[k % NK]);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r * NK / 8 == k) grad(8 + r);
      });
    };
    if (begin < steps) {
      sync(begin);
#pragma unroll
      for (int k = 0; k < T::LOADS; ++k) tile.load(k);
    }
    int n = begin + 1;
    const int some = min(steps, max(begin, whole)) + 1;
    for (; n < some; ++n) turn(n, std::true_type{});
    for (; n <= steps; ++n) turn(n, std::false_type{});
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    if (!live) return;
    const long long part = ((long long)h * a.Tk + seq.k0 + key) * a.dr;
#pragma unroll
    for (int d = 0; d < NK; ++d) {
      const int c = 32 * (d < NT ? d : d - NT);
      store_tile(d < NT ? dkv : dr_part, (d < NT ? row * (a.dn + a.dv) : part) + c, d < NT && g_bf16, dk[d], a.scale,
                 half, (d < NT ? a.dn : a.dr) - c);
    }
  }
}

// dr = the heads' parts added in their order; rows outside the sequences stay.
// 4096 tokens, 128 heads: 22 us for 134 MB of parts, 6 TB/s.
__global__ __launch_bounds__(256) void k_attn_dr(const float* __restrict__ part, const int32_t* __restrict__ cu_k,
                                                 int B, long long Tk, int dr, int H, void* out, bool bf16) {
  const long long n = Tk * dr / 4, i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const long long t = i / (dr / 4);
  if (t < cu_k[0] || t >= cu_k[B]) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* p = reinterpret_cast<const float4*>(part) + i;
#pragma unroll 8
  for (int h = 0; h < H; ++h) {
    const float4 v = p[h * n];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  store4(out, 4 * i, bf16, s.x, s.y, s.z, s.w);
}

size_t stat_bytes(long long Tq, int H) { return (size_t)ceil_div(Tq * H, 32) * 256; }

}  // namespace

size_t attention_backward_workspace_bytes(long long Tq, long long Tk, int H, int dr) {
  if (Tq < 0 || Tk < 0 || Tq >= (1LL << 31) || Tk >= (1LL << 31) || H < 1 || H > 1024 || dr < 8 || dr > MLA_MAX_DR ||
      dr % 8)
    return 0;
  return stat_bytes(Tq, H) + (size_t)H * Tk * dr * sizeof(float);
}

moe_status attention_backward(const void* dout, const void* q, const void* kv, const void* k_rope, long long ldr,
                              const void* out, moe_dtype out_t, const float* lse, const int32_t* cu_q,
                              const int32_t* cu_k, int B, long long Tq, long long Tk, int H, int dn, int dr, int dv,
                              bool causal, float scale, void* dq, void* dkv, void* dk_rope, moe_dtype g_t, void* ws,
                              size_t ws_bytes, void* stream) {
  moe_status st = attn_check(__func__, q, kv, k_rope, ldr, cu_q, cu_k, B, Tq, Tk, H, dn, dr, dv, scale);
  if (st != MOE_OK) return st;
  MOE_REQUIRE((out_t == MOE_F32 || out_t == MOE_BF16) && (g_t == MOE_F32 || g_t == MOE_BF16), MOE_EINVAL,
              "out_t and g_t must be MOE_F32 or MOE_BF16");
  if (B == 0 || (Tq == 0 && Tk == 0)) return MOE_OK;
  MOE_REQUIRE(cu_q && cu_k && (Tq == 0 || (q && dout && out && lse && dq)) && (Tk == 0 || (kv && k_rope && dkv && dk_rope)),
              MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(dout) && aligned16(out) && aligned16(dq) && aligned16(dkv) && aligned16(dk_rope) &&
                  aligned16(ws) && aligned4(lse),
              MOE_EINVAL, "dout, out, the gradients and ws must be 16-byte aligned");
  MOE_REQUIRE(ws && ws_bytes >= attention_backward_workspace_bytes(Tq, Tk, H, dr), MOE_EWORKSPACE,
              "workspace smaller than mla_attention_backward_workspace_bytes");
  float* stat = static_cast<float*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + stat_bytes(Tq, H));
  hipStream_t s = as_stream(stream);
  const uint16_t* g = static_cast<const uint16_t*>(dout);
  const bool bf16 = g_t == MOE_BF16;
  auto args = [&](bool by_key) {
    return attn_args(q, kv, k_rope, ldr, cu_q, cu_k, B, Tq, Tk, H, dn, dr, dv, causal, scale, 128, by_key);
  };
  auto go = [&](auto kq, auto kkv) {
    if (Tq > 0) {
      const AttnArgs a = args(false);
      hipLaunchKernelGGL(kq, dim3((unsigned)(8 * a.per_xcd)), dim3(256), 0, s, a, g, out, out_t == MOE_BF16, lse, dq,
                         bf16, stat);
    }
    if (Tk > 0) {
      const AttnArgs a = args(true);
      hipLaunchKernelGGL(kkv, dim3((unsigned)(8 * a.per_xcd)), dim3(512), 0, s, a, g, stat, dkv, bf16, part);
    }
  };
  // as in the forward: 2 sequences of about 2000, 32 heads of 64 + 32, 456 us for 642;
  // 8 of about 1000, 64 heads of 40 + 24, 623 for 827
  if (dn <= 64 && dr <= 32 && dv <= 64)
    go(k_attn_dq<64, 32, 64>, k_attn_dkv<64, 32, 64>);
  else
    go(k_attn_dq<128, 64, 128>, k_attn_dkv<128, 64, 128>);
  if (Tk > 0)
    hipLaunchKernelGGL(k_attn_dr, dim3((unsigned)ceil_div(Tk * dr / 4, 256)), dim3(256), 0, s, part, cu_k, B, Tk, dr, H,
                       dk_rope, bf16);
  return launch_status("mla_attention_backward");
}

}  // namespace moe
