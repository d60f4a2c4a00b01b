// moe_layer_few: the whole expert layer for up to MOE_FEW_TOKENS tokens.
//
//   s = sigmoid(u . e),  top-K of s + b,  g = s / sum of the selected s
//   out = resid + sum of the shared FFN(u) + sum_k g_k FFN_k(u)
// ("DeepSeek-V3 Technical Report" reading guide, xyznot.com, Method section
// 2: affinity sentence, gate equation, combine equation; SwiGLU FFNs.)
//
// With few tokens the layer is the reading of the touched experts' weights.
// Every product runs on the weight stream of skinny.h, 16 weight rows x 16
// tokens to a matrix instruction; a token that did not select an expert
// costs nothing there, since an expert's tokens are gathered first.
//
//   k_few_logits  partial logits, the K axis split over blocks; clears the
//                 counters of the kernels behind it
//   k_few_select  one block, a wave per token: scores, selection, gates, the
//                 list of the touched experts and their tokens.  The blocks
//                 beside it already run the shared experts' gate/up, which
//                 needs no selection.  Small layers do without this launch:
//                 there each block of k_few_up selects for itself
//   k_few_up      h = SiLU(W_gate x) (W_up x) of the touched experts, 16
//                 columns of h of one expert to a block
//   k_few_down    y = W_down h, fp32, 32 columns of one expert to a block; the
//                 last block of a column tile forms the gated sum in the order
//                 residual, shared, routed 0..K-1 (a launch of its own: 72
//                 against 69 us for the 4-bit layer and one token, 1330
//                 against 1343 for E4M3 and 32)
//
// "Last block": it counts the others' arrivals; nobody waits for anybody
// inside a kernel.  What such a block reads of the others' results was stored
// and is loaded at device scope, past the caches of one XCD, and each block
// counts itself after its stores have completed.
//
// Measured, d = 7168, I = 2048, 256 routed and one shared expert, K = 8: 4-bit
// weights and one token 64 us, of them logits 5, selection 8, gate/up 30 (4.2
// TB/s of weights), down 22 (3.2 TB/s), 32 tokens 815 us; bf16 and 4 tokens 481
// to 505 us (5.5 to 5.8 TB/s over the call, gate/up and down 6.0); E4M3 and 32
// tokens 1264 to 1336 us (5.4 to 5.7 TB/s).  The larger ones are bound by the
// weight stream, whose ceiling with every CU reading is about 6.1 TB/s; one
// token of 4-bit weights, 218 MB, by the chain of logits and selection and by
// the starts and tails of the two products.
//
// Measured against one persistent kernel behind the logits (blocks that take
// gate/up and then down items from queues, a down item waiting for its
// expert's gate/up items), on the products as they then were: 4-bit, one
// token, 75 us against 69; E4M3, 32 tokens, 1433 against 1343.  Its blocks end
// unevenly (a CU's older waves are served first: 12 us an item against 28 to
// 49), which the dispatch of fresh blocks evens out.
#include "skinny.h"
#include "vec8.h"

namespace moe {

namespace {

constexpr int FEW_T = MOE_FEW_TOKENS;
constexpr int FEW_W = 4;    // waves of a product block
constexpr int FEW_RT = 2;   // 16-row tiles of a product block
// Steps a product wave's loads run ahead, issued together: an E2M1 step takes
// half a cache line of a row (4-bit layer, 32 tokens, 812 us against 830 with a
// step at a time, one token 63.7 against 64.7; E4M3, 32 tokens, 1264 against
// 1281, each pair on one card; bf16 the same).
constexpr int FEW_D = 2;
constexpr int LOGIT_W = 8;  // waves of a router block
constexpr int FEW_THREADS = 64 * FEW_W;
constexpr int SELECT_W = 8;   // waves of a k_few_select block
constexpr int LOGIT_PARTS = 16;
// Words of a cache line: atomics of all XCDs on one line pass at 30 to 40 a
// microsecond, so busy counters have a line each.
constexpr int FEW_LINE = 32;

// Touched routed experts, in ascending order, and the tokens of each.
struct FewLists {
  int32_t* n;       // [1] touched routed experts
  int32_t* expert;  // [Nr]
  int32_t* tokens;  // [Nr] tokens of the expert
  int32_t* pair;    // [Nr, FEW_T] t << 16 | k of the expert's tokens, ascending
};

struct FewWs {
  uint32_t* column_done;  // [ceil(d / 32)] lines: down blocks done of each column tile
  int n_column_done;      // words
  float* z;  // [parts, T, Nr]
  FewLists lists;
  void* h;   // [T (K + Ns), I], row t (K + Ns) + k; shared expert j is k = K + j
  float* y;  // [T (K + Ns), d]
  size_t bytes;
};

// K axis parts of the router: enough blocks to occupy the chip, at least one
// step for every wave, and few enough that the selection can have all of a
// token's partial logits in flight at once.
int few_parts(int d, int Nr) {
  const int step = 4 * SkinnyWeight<MOE_F32>::EPL * SkinnyWeight<MOE_F32>::LD;
  const int tiles = (Nr + 15) / 16, steps = (d + step - 1) / step;
  int parts = 512 / tiles;
  if (parts > LOGIT_PARTS) parts = LOGIT_PARTS;
  if (parts > steps / LOGIT_W) parts = steps / LOGIT_W;
  return parts < 1 ? 1 : parts;
}

FewWs few_ws(void* base, int T, int d, int Nr, int Ns, int I, int K, moe_dtype u_t) {
  FewWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    at += (n + 255) / 256 * 256;
    return p;
  };
  const size_t pairs = (size_t)T * (K + Ns);
  const int columns = (d + FEW_RT * 16 - 1) / (FEW_RT * 16);
  w.n_column_done = columns * FEW_LINE;
  w.column_done = reinterpret_cast<uint32_t*>(take((size_t)w.n_column_done * 4));
  w.z = reinterpret_cast<float*>(take((size_t)few_parts(d, Nr) * T * Nr * 4));
  w.lists.n = reinterpret_cast<int32_t*>(take(4));
  w.lists.expert = reinterpret_cast<int32_t*>(take((size_t)Nr * 4));
  w.lists.tokens = reinterpret_cast<int32_t*>(take((size_t)Nr * 4));
  w.lists.pair = reinterpret_cast<int32_t*>(take((size_t)Nr * FEW_T * 4));
  w.h = take(pairs * I * (u_t == MOE_F32 ? 4 : 2));
  w.y = reinterpret_cast<float*>(take(pairs * d * 4));
  w.bytes = at;
  return w;
}

// --------------------------------------------------------------- routing --
template <typename UT, int NT>
__global__ __launch_bounds__(64 * LOGIT_W) void k_few_logits(const UT* __restrict__ u, const float* __restrict__ e,
                                                             int T, int d, int Nr, int steps_per_part,
                                                             float* __restrict__ z, uint32_t* __restrict__ ctl,
                                                             int n_ctl) {
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * 64 * LOGIT_W + threadIdx.x; i < n_ctl;
       i += gridDim.x * gridDim.y * 64 * LOGIT_W)
    ctl[i] = 0;
  using S = Skinny<MOE_F32, UT, 1, NT>;
  __shared__ sk_f32x4 red[LOGIT_W * NT * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = blockIdx.x * 16, part = blockIdx.y;
  typename S::Lanes L;
  L.K = d;
  L.g = lane >> 4;
  L.rw = sk_rsrc(e, (uint32_t)Nr * (uint32_t)d * 4u);
  L.rx = sk_rsrc(u, (uint32_t)T * (uint32_t)d * (uint32_t)sizeof(UT));
  const int r = e0 + (lane & 15);
  L.w_off[0] = r < Nr ? (uint32_t)r * (uint32_t)d * 4u + L.g * 16u : SK_OOB;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = n * 16 + (lane & 15);
    L.x_off[n] = t < T ? (uint32_t)t * (uint32_t)d * (uint32_t)sizeof(UT) + L.g * (uint32_t)S::XBYTES : SK_OOB;
  }
  const int steps = (d + S::STEP - 1) / S::STEP;
  const int s0 = part * steps_per_part;
  const int s1 = s0 + steps_per_part < steps ? s0 + steps_per_part : steps;
  sk_f32x4 acc[1][NT];
  S::template run_part<2>(acc, L, s0, s1, wave, LOGIT_W);
  sk_put<1, NT>(red, acc, threadIdx.x);
  for (int i = threadIdx.x; i < NT * 64; i += 64 * LOGIT_W) {
    const int l = i & 63, n = i >> 6, t = n * 16 + (l & 15);
    if (t >= T) continue;
    const sk_f32x4 s = sk_get<LOGIT_W, 1, NT>(red, 0, n, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ex = e0 + 4 * (l >> 4) + j;
      if (ex < Nr) z[((long long)part * T + t) * Nr + ex] = s[j];
    }
  }
}

template <typename V>
__device__ __forceinline__ void few_post(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void few_post4(float* p, sk_f32x4 v) {
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  few_post(q, (uint64_t)__float_as_uint(v[1]) << 32 | __float_as_uint(v[0]));
  few_post(q + 1, (uint64_t)__float_as_uint(v[3]) << 32 | __float_as_uint(v[2]));
}
__device__ __forceinline__ sk_f32x4 few_peek4(const float* p) {
  const uint64_t* q = reinterpret_cast<const uint64_t*>(p);
  const uint64_t a = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t b = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return sk_f32x4{__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)b),
                  __uint_as_float((uint32_t)(b >> 32))};
}

// Largest v of the wave (row shifts, then the rows' last lanes are passed on;
// lane 63 holds the result).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto mx = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));
  v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
  v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Routing of token t by one wave (EPL experts per lane, expert lane + 64 j):
// K times the largest order key of s + b among the experts not taken yet, a
// tie to the lowest index.  An expert's bit in `mask` gains the token.
template <int EPL>
__device__ __forceinline__ void few_route_token(const float* __restrict__ z, int parts, const float* __restrict__ bias,
                                                int t, int lane, int T, int Nr, int K,
                                                int32_t* topk_idx,
                                                float* topk_gate, float* topk_score, uint16_t* pick,
                                                uint32_t* mask, bool write) {
  float s[EPL];
  uint32_t key[EPL];
  uint32_t avail = 0;
  // partial logits, added in ascending order of the parts; read without
  // branches (past Nr: expert Nr - 1), so their latencies overlap
  constexpr int AHEAD = EPL > 4 ? 1 : LOGIT_PARTS;
  int at[EPL];
  float add[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int i = lane + 64 * j < Nr ? lane + 64 * j : Nr - 1;
    s[j] = 0.f;
    at[j] = t * Nr + i;
    add[j] = bias[i];
  }
  for (int p0 = 0; p0 < parts; p0 += AHEAD) {
    float v[AHEAD][EPL];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[q][j] = z[(p0 + q < parts ? p0 + q : p0) * T * Nr + at[j]];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] += p0 + q < parts ? v[q][j] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int i = lane + 64 * j;
    key[j] = 0;
    s[j] = 1.0f / (1.0f + expf(-s[j]));
    if (i < Nr) {
      key[j] = float_order_key(s[j] + add[j]);
      avail |= 1u << j;
    }
  }
  int my_idx = 0;
  float my_s = 0.f, sum = 0.f;
  for (int k = 0; k < K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if ((avail >> j & 1) && key[j] > best) best = key[j];
    const uint32_t top = wave_max_u32(best);
    int pick = -1;
    float sk = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const unsigned long long b = __ballot((avail >> j & 1) && key[j] == top);
      if (pick < 0 && b) {
        const int owner = __builtin_ctzll(b);
        pick = owner + 64 * j;
        sk = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s[j]), owner));
        if (lane == owner) avail &= ~(1u << j);
      }
    }
    if (lane == k) {
      my_idx = pick;
      my_s = sk;
    }
    sum += sk;
  }
  if (lane < K) {
    const int o = t * K + lane;
    pick[o] = (uint16_t)my_idx;
    atomicOr(&mask[my_idx], 1u << t);
    if (write) {
      topk_idx[o] = my_idx;
      topk_gate[o] = my_s / sum;
      if (topk_score) topk_score[o] = my_s;
    }
  }
}

__global__ void k_few_no_load(int32_t* load, int Nr) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < Nr) load[i] = 0;
}

// -------------------------------------------------- selection, products --
struct FewArgs {
  const void* u;  // [T, d]
  const void* w13;
  const void* w13_scale;
  const void* w2;
  const void* w2_scale;
  const float* z;
  const float* bias;
  const void* resid;  // [T, d] or NULL
  int32_t* topk_idx;
  float* topk_gate;
  float* topk_score;
  int32_t* load;
  void* h;
  float* y;
  void* out;  // [T, d]
  uint32_t* column_done;
  FewLists lists;
  int T, d, Nr, Ns, I, K, parts;
  bool resid_bf16, out_bf16;
};

// The block's device-scope stores have completed, and the counter has counted
// them.  Returns the counter's value before, to every thread.
__device__ __forceinline__ uint32_t few_signal(uint32_t* counter, uint32_t* shared, int tid) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0)
    *shared = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return *shared;
}

struct FewSelect {
  uint32_t mask[MOE_MAX_EXPERTS];     // tokens of each expert
  uint16_t place[MOE_MAX_EXPERTS];    // its place in the list
  uint16_t pick[FEW_T * MOE_MAX_K];   // [T, K] selected experts
  int n, wanted;                      // touched experts, and the one at the wanted place of the list
};

// Selection by a block of W waves.  write: the outputs and the lists are stored.
template <int W>
__device__ __forceinline__ void few_select(const FewArgs& A, FewSelect& S, int tid, bool write, int want) {
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < A.Nr; e += 64 * W) S.mask[e] = 0;
  __syncthreads();
  for (int t = wave; t < A.T; t += W) {
    if (A.Nr <= 64)
      few_route_token<1>(A.z, A.parts, A.bias, t, lane, A.T, A.Nr, A.K, A.topk_idx, A.topk_gate, A.topk_score, S.pick,
                         S.mask, write);
    else if (A.Nr <= 256)
      few_route_token<4>(A.z, A.parts, A.bias, t, lane, A.T, A.Nr, A.K, A.topk_idx, A.topk_gate, A.topk_score, S.pick,
                         S.mask, write);
    else
      few_route_token<16>(A.z, A.parts, A.bias, t, lane, A.T, A.Nr, A.K, A.topk_idx, A.topk_gate, A.topk_score, S.pick,
                          S.mask, write);
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < A.Nr; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t m = e < A.Nr ? S.mask[e] : 0u;
      const unsigned long long b = __ballot(m != 0);
      const int at = n + __popcll(b & ((1ull << lane) - 1));
      if (m) {
        S.place[e] = (uint16_t)at;
        if (at == want) S.wanted = e;
        if (write) {
          A.lists.expert[at] = e;
          A.lists.tokens[at] = __popc(m);
        }
      }
      n += __popcll(b);
    }
    if (lane == 0) {
      S.n = n;
      if (write) *A.lists.n = n;
    }
  }
  if (write && A.load)
    for (int e = tid; e < A.Nr; e += 64 * W) A.load[e] = __popc(S.mask[e]);
  __syncthreads();
  if (!write) return;
  for (int q = tid; q < A.T * A.K; q += 64 * W) {
    const int t = q / A.K, e = S.pick[q];
    A.lists.pair[S.place[e] * FEW_T + __popc(S.mask[e] & ((1u << t) - 1))] = t << 16 | (q - t * A.K);
  }
}

// One item: 16 RT weight rows of one expert (gate/up: 8 RT gate rows and the
// up rows of the same columns of h) on up to 16 of its tokens, j0 and on.
// p: token and slot of the lane's token column.
template <int WT, typename XT, bool UP, bool SV, int W, bool PK>
__device__ __forceinline__ void few_product(const FewArgs& A, int ex, int toks, int j0, int p, int col0,
                                            sk_f32x4* red, int tid) {
  constexpr int RT = FEW_RT;
  using S = Skinny<WT, XT, RT, 1, SV, PK>;
  const int Kd = UP ? A.d : A.I, Nd = UP ? A.I : A.d;
  const int lane = tid & 63, wave = tid >> 6;
  const int R = A.K + A.Ns;  // h and y rows of a token
  const int wrows = UP ? 2 * Nd : Nd;
  const uint32_t row_bytes = (uint32_t)sk_row_bytes(WT, Kd);
  const void* scale = UP ? A.w13_scale : A.w2_scale;
  typename S::Lanes L;
  L.K = Kd;
  L.g = lane >> 4;
  L.rw = sk_rsrc(static_cast<const uint8_t*>(UP ? A.w13 : A.w2) + (long long)ex * wrows * row_bytes,
                 (uint32_t)wrows * row_bytes);
  L.rx = sk_rsrc(UP ? A.u : A.h, (uint32_t)(UP ? A.T : A.T * R) * (uint32_t)Kd * (uint32_t)sizeof(XT));
  const uint32_t s_row = (uint32_t)Kd / 32u;
  if (WT == MOE_E2M1)
    L.rs = sk_rsrc(static_cast<const uint8_t*>(scale) + (long long)ex * wrows * s_row, (uint32_t)wrows * s_row);
  if (WT == MOE_E4M3) {
    const int nk = Kd / 128;
    const float* sc = static_cast<const float*>(scale) + (long long)ex * (wrows / 128) * nk;
    L.blk_lo = sc + (long long)(col0 / 128) * nk;
    L.blk_hi = sc + (long long)((UP ? Nd + col0 : col0) / 128) * nk;
  }
#pragma unroll
  for (int f = 0; f < RT; ++f) {
    const int c = col0 + (UP ? f % (RT / 2) : f) * 16 + (lane & 15);
    const uint32_t r = (uint32_t)(UP && f >= RT / 2 ? Nd + c : c);
    L.w_off[f] = c < Nd ? r * row_bytes + L.g * 16u : SK_OOB;
    L.s_off[f] = c < Nd ? r * s_row + (SV ? 0 : L.g) : SK_OOB;
  }
  const int j = PK ? (lane & 15) / S::XV : lane & 15;  // the token whose x the lane reads
  const int px = PK ? __shfl(p, j, 64) : p;
  const uint32_t x_row = (uint32_t)(UP ? px >> 16 : (px >> 16) * R + (px & 0xFFFF));
  L.x_off[0] = j0 + j < toks ? x_row * (uint32_t)Kd * (uint32_t)sizeof(XT) + L.g * (uint32_t)S::XBYTES +
                                   (PK ? (uint32_t)(lane % S::XV) * 16u : 0u)
                             : SK_OOB;
  sk_f32x4 acc[RT][S::AC];
  S::template run_part<FEW_D, FEW_D>(acc, L, 0, (Kd + S::STEP - 1) / S::STEP, wave, W);
  if constexpr (PK)
    sk_put_packed<RT, S::XV>(red, acc, tid);
  else
    sk_put<RT, 1>(red, acc, tid);
  auto sum = [&](int f) {
    if constexpr (PK)
      return sk_get_packed<W, RT, S::XV>(red, f, lane);
    else
      return sk_get<W, RT, 1>(red, f, 0, lane);
  };
  const int hr = (p >> 16) * R + (p & 0xFFFF);  // row of h or y of the lane's token
  constexpr int OUT_TILES = UP ? RT / 2 : RT;
  for (int i = tid; i < OUT_TILES * 64; i += 64 * W) {
    const int f = i >> 6, c = col0 + f * 16 + 4 * L.g;  // 64 threads to a tile: each its own lane's column
    if (!S::holds(lane, j0, toks) || c >= Nd) continue;  // Nd % 4 == 0: four columns exist or none
    const long long o = (long long)hr * Nd + c;
    const sk_f32x4 a = sum(f);
    if constexpr (UP) {
      const sk_f32x4 b = sum(f + RT / 2);
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = silu(a[q]) * b[q];
      if constexpr (sizeof(XT) == 4) {
        *reinterpret_cast<sk_f32x4*>(static_cast<float*>(A.h) + o) = sk_f32x4{v[0], v[1], v[2], v[3]};
      } else {
        // h is rounded to bf16, as the operand of the down projection's
        // matrix instructions (fp32 layers keep it in fp32).  It is what sets
        // these layers apart from one with an fp32 h, whose result they are
        // 1.3e-3 to 2.3e-3 of its norm from (u added, both in bf16); with h
        // rounded there too, 0 to 2e-4
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.h) + o) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    } else {
      few_post4(A.y + o, a);
    }
  }
}

__device__ __forceinline__ sk_f32x4 few_load4(const void* p, bool bf16, long long i) {
  if (!bf16) return *reinterpret_cast<const sk_f32x4*>(static_cast<const float*>(p) + i);
  const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  return sk_f32x4{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u), __uint_as_float(q.y << 16),
                  __uint_as_float(q.y & 0xFFFF0000u)};
}

// out[:, col0 .. col0 + 31], eight threads to a token.
__device__ __forceinline__ void few_combine(const FewArgs& A, int col0, int tid) {
  constexpr int PER = FEW_RT * 4;  // threads to a token, four columns each
  const int t = tid / PER, c = col0 + (tid % PER) * 4;
  if (c >= A.d) return;
  for (int tt = t; tt < A.T; tt += FEW_THREADS / PER) {
    const long long o = (long long)tt * A.d + c;
    const float* y = A.y + (long long)tt * (A.K + A.Ns) * A.d + c;
    sk_f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (A.resid) s = few_load4(A.resid, A.resid_bf16, o);
    for (int j = 0; j < A.Ns; ++j) s += few_peek4(y + (long long)(A.K + j) * A.d);
    for (int k0 = 0; k0 < A.K; k0 += 4) {
      sk_f32x4 v[4];
      float g[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int kk = k0 + k < A.K ? k0 + k : k0;
        v[k] = few_peek4(y + (long long)kk * A.d);
        g[k] = A.topk_gate[tt * A.K + kk];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k0 + k < A.K)
#pragma unroll
          for (int q = 0; q < 4; ++q) s[q] = fmaf(g[k], v[k][q], s[q]);
    }
    if (A.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.out) + o) =
          make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    else
      *reinterpret_cast<sk_f32x4*>(static_cast<float*>(A.out) + o) = s;
  }
}

// An expert's column tile on all its tokens, as many at a time as the form
// takes; the rows are read again from a cache that has just held them.
template <int WT, typename XT, bool UP, bool SV, bool PK, int W>
__device__ __forceinline__ void few_item(const FewArgs& A, int ex, int toks, const int32_t* pairs, int p, int col0,
                                         sk_f32x4* red, int tid) {
  constexpr int TOKENS = Skinny<WT, XT, FEW_RT, 1, SV, PK>::TOKENS;
  for (int j0 = 0; j0 < toks; j0 += TOKENS) {
    if (j0) {
      const int j = j0 + (tid & 15);
      p = !pairs ? p + (TOKENS << 16) : pairs[j < FEW_T ? j : FEW_T - 1];
      __syncthreads();  // red is read until here
    }
    few_product<WT, XT, UP, SV, W, PK>(A, ex, toks, j0, p, col0, red, tid);
  }
}

constexpr int FEW_UP_COLS = FEW_RT * 8, FEW_DOWN_COLS = FEW_RT * 16;  // columns of a block

// Block 0 selects; the others are the shared experts' gate/up, with many
// waves to a block: they are alone on the chip.
template <int WT, typename XT, bool SV, bool PK>
__global__ __launch_bounds__(64 * SELECT_W) void k_few_select(FewArgs A) {
  __shared__ union {
    sk_f32x4 red[SELECT_W * FEW_RT * 64];
    FewSelect select;
  } lds;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    few_select<SELECT_W>(A, lds.select, tid, true, -1);
    return;
  }
  const int tiles = (A.I + FEW_UP_COLS - 1) / FEW_UP_COLS;
  const int item = blockIdx.x - 1, e = item / tiles;
  few_item<WT, XT, true, SV, PK, SELECT_W>(A, A.Nr + e, A.T, nullptr, (tid & 15) << 16 | (A.K + e), (item % tiles) * FEW_UP_COLS,
                             lds.red, tid);
}

// SELF: there was no k_few_select.  Every block of a routed expert selects for
// itself, the first one stores the results, and the shared experts' blocks
// come in front.
template <int WT, typename XT, bool SV, bool PK, bool SELF>
__global__ __launch_bounds__(FEW_THREADS, PK ? 4 : 1) void k_few_up(FewArgs A) {
  __shared__ union {
    sk_f32x4 red[FEW_W * FEW_RT * 64];
    FewSelect select;
  } lds;
  __shared__ int32_t s_pair[FEW_T];
  const int tid = threadIdx.x;
  const int tiles = (A.I + FEW_UP_COLS - 1) / FEW_UP_COLS, e = blockIdx.x / tiles;
  int ex, toks, p;
  const int32_t* pairs;
  if constexpr (!SELF) {
    // one memory latency for all four; what lies past the list is not used
    const int n = *A.lists.n;
    ex = A.lists.expert[e];
    toks = A.lists.tokens[e];
    pairs = A.lists.pair + e * FEW_T;
    p = pairs[tid & 15];
    if (e >= n) return;
  } else if (e < A.Ns) {
    ex = A.Nr + e;
    toks = A.T;
    pairs = nullptr;
    p = (tid & 15) << 16 | (A.K + e);
  } else {
    few_select<FEW_W>(A, lds.select, tid, (int)blockIdx.x == A.Ns * tiles, e - A.Ns);
    if (e - A.Ns >= lds.select.n) return;
    ex = __builtin_amdgcn_readfirstlane(lds.select.wanted);
    const uint32_t m = __builtin_amdgcn_readfirstlane(lds.select.mask[ex]);
    toks = __popc(m);
    for (int q = tid; q < A.T * A.K; q += FEW_THREADS) {
      const int t = q / A.K;
      if (lds.select.pick[q] == ex) s_pair[__popc(m & ((1u << t) - 1))] = t << 16 | (q - t * A.K);
    }
    __syncthreads();  // red lies on the selection
    pairs = s_pair;
    p = pairs[tid & 15];
  }
  few_item<WT, XT, true, SV, PK, FEW_W>(A, ex, toks, pairs, p, (blockIdx.x % tiles) * FEW_UP_COLS, lds.red, tid);
}

template <int WT, typename XT, bool SV, bool PK>
__global__ __launch_bounds__(FEW_THREADS, PK ? 4 : 1) void k_few_down(FewArgs A) {
  __shared__ sk_f32x4 red[FEW_W * FEW_RT * 64];
  __shared__ uint32_t s_count;
  const int tid = threadIdx.x;
  const int tiles = (A.d + FEW_DOWN_COLS - 1) / FEW_DOWN_COLS, e = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int n = *A.lists.n;
  int ex = A.Nr + e, toks = A.T, p = (tid & 15) << 16 | (A.K + e);
  const int32_t* pairs = nullptr;
  if (e >= A.Ns) {  // the shared experts come first: they have the most tokens
    ex = A.lists.expert[e - A.Ns];
    toks = A.lists.tokens[e - A.Ns];
    pairs = A.lists.pair + (e - A.Ns) * FEW_T;
    p = pairs[tid & 15];
    if (e - A.Ns >= n) return;
  }
  few_item<WT, XT, false, SV, PK, FEW_W>(A, ex, toks, pairs, p, tile * FEW_DOWN_COLS, red, tid);
  if (few_signal(A.column_done + tile * FEW_LINE, &s_count, tid) == (uint32_t)(A.Ns + n) - 1)
    few_combine(A, tile * FEW_DOWN_COLS, tid);
}

// Whether the gate/up blocks select for themselves, which saves a launch and
// costs every block the selection of T / FEW_W tokens by each wave, in length
// about as the experts of a lane.  In us, with k_few_select and without: fp32, d
// = 256, 16 + 1 experts, one token 18.2 / 15.6, 8 tokens 19.3 / 16.6, 32 23.3 /
// 25.7; bf16, d = 2048, I = 1408, 64 + 2 experts, one token 44 / 39, 2 65 / 61,
// 4 90 / 88, 8 126 / 132; 4-bit, d = 7168, 256 + 1 experts, one token, I = 512
// 33.0 / 31.6, I = 2048 64.7 / 67.7, with 64 + 1 experts 64.4 / 63.3.
bool few_selects_for_itself(const FewArgs& A, int blocks) {
  const int lane = A.Nr <= 64 ? 1 : A.Nr <= 256 ? 4 : 16, tokens = (A.T + FEW_W - 1) / FEW_W;
  return A.T <= 2 * FEW_W && blocks * tokens * lane <= 2560;
}

// Packed where an expert has few tokens: at most two for every routed expert
// on average, or no more tokens than fit.  (d = 7168, 256 experts, whole
// layer: E4M3, 32 tokens, 1285 us against 1330; 4-bit, one token, 66 against
// 69, with the registers held to four waves a SIMD, else 71; the form that
// selects for itself spills 11 of them, 48 bytes of scratch a lane.)  With more
// tokens an expert the repeated reading of its rows would cost more than the
// loads of x that it saves.
template <int WT, typename XT, bool SV>
void launch_blocks(const FewArgs& A, hipStream_t st) {
  constexpr bool NARROW = WT == MOE_E4M3 || WT == MOE_E2M1;
  constexpr int PACKED = Skinny<WT, XT, FEW_RT, 1, SV, NARROW>::TOKENS;
  const int touched = A.T * A.K < A.Nr ? A.T * A.K : A.Nr;
  const int up = (A.I + FEW_UP_COLS - 1) / FEW_UP_COLS, down = (A.d + FEW_DOWN_COLS - 1) / FEW_DOWN_COLS;
  const dim3 block(FEW_THREADS);
  auto select = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(1 + A.Ns * up), dim3(64 * SELECT_W), 0, st, A); };
  const bool self = few_selects_for_itself(A, (touched + A.Ns) * up);
  auto products = [&](auto k_up, auto k_self, auto k_down) {
    if (self)
      hipLaunchKernelGGL(k_self, dim3((touched + A.Ns) * up), block, 0, st, A);
    else
      hipLaunchKernelGGL(k_up, dim3(touched * up), block, 0, st, A);
    hipLaunchKernelGGL(k_down, dim3((touched + A.Ns) * down), block, 0, st, A);
  };
  if (!self) {
    if (NARROW && A.T <= PACKED)
      select(k_few_select<WT, XT, SV, NARROW>);
    else
      select(k_few_select<WT, XT, SV, false>);
  }
  if (NARROW && (A.T <= PACKED || A.T * A.K <= 2 * A.Nr))
    products(k_few_up<WT, XT, SV, NARROW, false>, k_few_up<WT, XT, SV, NARROW, true>, k_few_down<WT, XT, SV, NARROW>);
  else
    products(k_few_up<WT, XT, SV, false, false>, k_few_up<WT, XT, SV, false, true>, k_few_down<WT, XT, SV, false>);
}

template <int WT, typename XT>
void launch_layer(const FewArgs& A, hipStream_t st) {
  // rows of exponent bytes in whole words: read 16 at a time
  if (WT == MOE_E2M1 && A.d % 128 == 0 && A.I % 128 == 0 && aligned4(A.w13_scale) && aligned4(A.w2_scale))
    launch_blocks<WT, XT, WT == MOE_E2M1>(A, st);
  else
    launch_blocks<WT, XT, false>(A, st);
}

template <typename UT>
void launch_logits(const void* u, const float* e, int T, int d, int Nr, int parts, float* z, uint32_t* ctl, int n_ctl,
                   hipStream_t st) {
  const int step = Skinny<MOE_F32, UT, 1, 1>::STEP, steps = (d + step - 1) / step;
  const int per = (steps + parts - 1) / parts;
  const dim3 grid((Nr + 15) / 16, parts);
  if (T <= 16)
    hipLaunchKernelGGL((k_few_logits<UT, 1>), grid, dim3(64 * LOGIT_W), 0, st, static_cast<const UT*>(u), e, T, d, Nr,
                       per, z, ctl, n_ctl);
  else
    hipLaunchKernelGGL((k_few_logits<UT, 2>), grid, dim3(64 * LOGIT_W), 0, st, static_cast<const UT*>(u), e, T, d, Nr,
                       per, z, ctl, n_ctl);
}

bool few_sizes_ok(int T, int d, int Nr, int Ns, int I, int K) {
  return T >= 0 && T <= FEW_T && d >= 8 && d % 8 == 0 && I >= 8 && I % 8 == 0 && Nr >= 1 && Ns >= 0 &&
         Nr <= MOE_MAX_EXPERTS && Ns <= MOE_MAX_EXPERTS - Nr && K >= 1 && K <= MOE_MAX_K && K <= Nr;
}

}  // namespace

size_t layer_few_workspace_bytes(int T, int d, int Nr, int Ns, int I, int K, moe_dtype u_t) {
  if (!few_sizes_ok(T, d, Nr, Ns, I, K)) return 0;
  return few_ws(nullptr, T, d, Nr, Ns, I, K, u_t).bytes;
}

moe_status layer_few(const void* u, moe_dtype u_t, const float* centroids, const float* bias, moe_dtype w_t,
                     const void* w13, const void* w13_scale, const void* w2, const void* w2_scale, int T, int d, int Nr,
                     int Ns, int I, int K, const void* resid, moe_dtype r_t, int32_t* topk_idx, float* topk_gate,
                     float* topk_score, int32_t* expert_load, void* ws, size_t ws_bytes, void* out, moe_dtype out_t,
                     void* stream) {
  MOE_REQUIRE(u_t == MOE_F32 || u_t == MOE_BF16, MOE_EINVAL, "u_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(w_t == MOE_F32 || w_t == MOE_BF16 || w_t == MOE_E4M3 || w_t == MOE_E2M1, MOE_EINVAL, "bad w_t");
  MOE_REQUIRE(out_t == MOE_F32 || out_t == MOE_BF16, MOE_EINVAL, "out_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(!resid || r_t == MOE_F32 || r_t == MOE_BF16, MOE_EINVAL, "r_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(T >= 0 && d >= 8 && d % 8 == 0 && I >= 8 && I % 8 == 0, MOE_EINVAL,
              "need T >= 0, and d and I positive multiples of 8");
  MOE_REQUIRE(Nr >= 1 && Ns >= 0 && Nr <= MOE_MAX_EXPERTS && Ns <= MOE_MAX_EXPERTS - Nr, MOE_EINVAL,
              "Nr or Ns out of range");
  MOE_REQUIRE(K >= 1 && K <= MOE_MAX_K && K <= Nr, MOE_EINVAL, "K out of range");
  MOE_REQUIRE(T <= FEW_T, MOE_EUNSUPPORTED, "more than MOE_FEW_TOKENS tokens");
  MOE_REQUIRE((u_t == MOE_F32) == (w_t == MOE_F32), MOE_EUNSUPPORTED, "unsupported (u_t, w_t) combination");
  MOE_REQUIRE(w_t != MOE_E4M3 || (d % 128 == 0 && I % 128 == 0), MOE_EUNSUPPORTED,
              "E4M3 weights need d and I to be multiples of 128");
  MOE_REQUIRE(w_t != MOE_E2M1 || (d % 32 == 0 && I % 32 == 0), MOE_EUNSUPPORTED,
              "E2M1 weights need d and I to be multiples of 32");
  MOE_REQUIRE(fits31(2ull * I * sk_row_bytes(w_t, d)) && fits31((unsigned long long)d * sk_row_bytes(w_t, I)) &&
                  fits31((unsigned long long)Nr * d * 4) && fits31((unsigned long long)FEW_T * d * 4) &&
                  fits31((unsigned long long)FEW_T * (K + Ns) * I * 4),
              MOE_EUNSUPPORTED, "an expert's matrix, the centroids or h of 2 GiB or more");
  // blocks of at most 512 threads: a launch has fewer than 2^32
  const long long experts = (T * K < Nr ? T * K : Nr) + (long long)Ns;
  MOE_REQUIRE(experts * ceil_div(I, FEW_RT * 8) < (1 << 22) && experts * ceil_div(d, FEW_RT * 16) < (1 << 22),
              MOE_EUNSUPPORTED, "too many experts for I or d");
  if (T == 0) {
    if (!expert_load) return MOE_OK;
    hipLaunchKernelGGL(k_few_no_load, dim3((Nr + 255) / 256), dim3(256), 0, as_stream(stream), expert_load, Nr);
    return launch_status("moe_layer_few");
  }
  MOE_REQUIRE(u && centroids && bias && w13 && w2 && topk_idx && topk_gate && out, MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE((w_t != MOE_E4M3 && w_t != MOE_E2M1) || (w13_scale && w2_scale), MOE_EINVAL,
              "E4M3 and E2M1 weights need scales");
  MOE_REQUIRE(aligned16(u) && aligned16(centroids) && aligned16(w13) && aligned16(w2) && aligned16(resid) &&
                  aligned16(ws) && aligned16(out),
              MOE_EINVAL, "u, centroids, w13, w2, resid, ws and out must be 16-byte aligned");
  MOE_REQUIRE(ws && ws_bytes >= layer_few_workspace_bytes(T, d, Nr, Ns, I, K, u_t), MOE_EWORKSPACE,
              "workspace smaller than moe_layer_few_workspace_bytes");
  hipStream_t st = as_stream(stream);
  const FewWs w = few_ws(ws, T, d, Nr, Ns, I, K, u_t);
  const int parts = few_parts(d, Nr);
  if (u_t == MOE_F32)
    launch_logits<float>(u, centroids, T, d, Nr, parts, w.z, w.column_done, w.n_column_done, st);
  else
    launch_logits<uint16_t>(u, centroids, T, d, Nr, parts, w.z, w.column_done, w.n_column_done, st);
  const FewArgs A{u,          w13,        w13_scale,   w2,  w2_scale, w.z, bias,  resid,   topk_idx, topk_gate,
                  topk_score, expert_load, w.h,        w.y, out,      w.column_done, w.lists, T, d, Nr,
                  Ns,         I,          K,           parts, r_t == MOE_BF16, out_t == MOE_BF16};
  switch (w_t) {
    case MOE_F32: launch_layer<MOE_F32, float>(A, st); break;
    case MOE_BF16: launch_layer<MOE_BF16, uint16_t>(A, st); break;
    case MOE_E4M3: launch_layer<MOE_E4M3, uint16_t>(A, st); break;
    default: launch_layer<MOE_E2M1, uint16_t>(A, st); break;
  }
  return launch_status("moe_layer_few");
}

}  // namespace moe
