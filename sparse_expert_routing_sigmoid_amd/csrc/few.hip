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
//   k_few_logits  partial logits, the K axis split over blocks
//   k_few_select  one wave per token: scores, selection, gates; then the list
//                 of touched experts with their tokens
//   k_few_gate_up h = SiLU(W_gate x) (W_up x) of every (expert, token) pair
//   k_few_down    y = W_down h of every pair, fp32
//   k_few_combine the gated sum, in the order residual, shared, routed 0..K-1
#include "skinny.h"
#include "vec8.h"

namespace moe {

namespace {

constexpr int FEW_T = MOE_FEW_TOKENS;
constexpr int FEW_W = 4;    // waves of a product block
constexpr int FEW_RT = 2;   // 16-row tiles of a product block
constexpr int FEW_D = 2;    // steps a product wave's loads run ahead
constexpr int LOGIT_W = 8;  // waves of a router block
constexpr int LOGIT_PARTS = 8;

// Touched routed experts, in ascending order, and the tokens of each.
struct FewLists {
  int32_t* n;       // [1] touched routed experts
  int32_t* expert;  // [Nr]
  int32_t* tokens;  // [Nr] tokens of the expert
  int32_t* pair;    // [Nr, FEW_T] t << 16 | k of the expert's tokens, ascending
};

struct FewWs {
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
  int parts = 256 / tiles;
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
                                                             float* __restrict__ z) {
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
  sk_put<1, NT>(red, acc);
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
                                                int t, int T, int Nr, int K, int32_t* __restrict__ topk_idx,
                                                float* __restrict__ topk_gate, float* __restrict__ topk_score,
                                                uint32_t* mask) {
  const int lane = threadIdx.x & 63;
  float s[EPL];
  uint32_t key[EPL];
  uint32_t avail = 0;
  // partial logits, added in ascending order of the parts; read without
  // branches (past Nr: expert Nr - 1), so their latencies overlap
  constexpr int AHEAD = EPL > 4 ? 1 : LOGIT_PARTS;
  int at[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    s[j] = 0.f;
    at[j] = t * Nr + (lane + 64 * j < Nr ? lane + 64 * j : Nr - 1);
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
      key[j] = float_order_key(s[j] + bias[i]);
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
    topk_idx[o] = my_idx;
    topk_gate[o] = my_s / sum;
    if (topk_score) topk_score[o] = my_s;
    atomicOr(&mask[my_idx], 1u << t);
  }
}

template <int EPL>
__global__ __launch_bounds__(1024) void k_few_select(const float* __restrict__ z, int parts,
                                                     const float* __restrict__ bias, int T, int Nr, int K,
                                                     int32_t* __restrict__ topk_idx, float* __restrict__ topk_gate,
                                                     float* __restrict__ topk_score, int32_t* __restrict__ load,
                                                     FewLists lists) {
  __shared__ uint32_t mask[MOE_MAX_EXPERTS];  // tokens of each expert
  __shared__ int place[MOE_MAX_EXPERTS];      // its position in the list
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < Nr; i += 1024) mask[i] = 0;
  __syncthreads();
  for (int t = wave; t < T; t += 16)
    few_route_token<EPL>(z, parts, bias, t, T, Nr, K, topk_idx, topk_gate, topk_score, mask);
  __threadfence_block();  // topk_idx is read back below
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int i0 = 0; i0 < Nr; i0 += 64) {
      const int i = i0 + lane;
      const bool touched = i < Nr && mask[i] != 0;
      const unsigned long long b = __ballot(touched);
      const int at = n + __popcll(b & ((1ull << lane) - 1));
      if (touched) {
        place[i] = at;
        lists.expert[at] = i;
        lists.tokens[at] = __popc(mask[i]);
      }
      n += __popcll(b);
    }
    if (lane == 0) *lists.n = n;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * K; i += 1024) {
    const int t = i / K, k = i % K, ex = topk_idx[i];
    lists.pair[place[ex] * FEW_T + __popc(mask[ex] & ((1u << t) - 1))] = t << 16 | k;
  }
  if (load)
    for (int i = threadIdx.x; i < Nr; i += 1024) load[i] = __popc(mask[i]);
}

__global__ void k_few_no_load(int32_t* load, int Nr) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < Nr) load[i] = 0;
}

// -------------------------------------------------------------- products --
struct FewArgs {
  const void* x;      // gate/up: tokens u [T, Kd]; down: h [T (K + Ns), Kd]
  const void* w;      // [Nr + Ns, rows, Kd] as stored
  const void* scale;  // E4M3: fp32 [E, rows / 128, Kd / 128]; E2M1: bytes [E, rows, Kd / 32]
  void* out;          // gate/up: h [T (K + Ns), Nd]; down: y [T (K + Ns), Nd] fp32
  FewLists lists;
  int T, K, Nr, Ns, Nd, Kd;
};

// One item: 16 RT weight rows of one expert (gate/up: 8 RT gate rows and the
// up rows of the same columns of h) on up to 16 of its tokens, j0 and on.
template <int WT, typename XT, bool GATE_UP, bool SV>
__device__ __forceinline__ void few_item(const FewArgs& A, int ex, int toks, int j0, int p, int col0, sk_f32x4* red) {
  constexpr int RT = FEW_RT;
  using S = Skinny<WT, XT, RT, 1, SV>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int R = A.K + A.Ns;  // h and y rows of a token
  const int t = p >> 16, hr = t * R + (p & 0xFFFF);  // the lane's token column: its token, and its row of h and y
  const int wrows = GATE_UP ? 2 * A.Nd : A.Nd;
  const uint32_t row_bytes = (uint32_t)sk_row_bytes(WT, A.Kd);
  typename S::Lanes L;
  L.K = A.Kd;
  L.g = lane >> 4;
  L.rw = sk_rsrc(static_cast<const uint8_t*>(A.w) + (long long)ex * wrows * row_bytes, (uint32_t)wrows * row_bytes);
  L.rx = sk_rsrc(A.x, (uint32_t)(GATE_UP ? A.T : A.T * R) * (uint32_t)A.Kd * (uint32_t)sizeof(XT));
  const uint32_t s_row = (uint32_t)A.Kd / 32u;
  if (WT == MOE_E2M1)
    L.rs = sk_rsrc(static_cast<const uint8_t*>(A.scale) + (long long)ex * wrows * s_row, (uint32_t)wrows * s_row);
  if (WT == MOE_E4M3) {
    const int nk = A.Kd / 128;
    const float* sc = static_cast<const float*>(A.scale) + (long long)ex * (wrows / 128) * nk;
    L.blk_lo = sc + (long long)(col0 / 128) * nk;
    L.blk_hi = sc + (long long)((GATE_UP ? A.Nd + col0 : col0) / 128) * nk;
  }
#pragma unroll
  for (int f = 0; f < RT; ++f) {
    const int c = col0 + (GATE_UP ? f % (RT / 2) : f) * 16 + (lane & 15);
    const uint32_t r = (uint32_t)(GATE_UP && f >= RT / 2 ? A.Nd + c : c);
    L.w_off[f] = c < A.Nd ? r * row_bytes + L.g * 16u : SK_OOB;
    L.s_off[f] = c < A.Nd ? r * s_row + (SV ? 0 : L.g) : SK_OOB;
  }
  L.x_off[0] = j0 + (lane & 15) < toks ? (uint32_t)(GATE_UP ? t : hr) * (uint32_t)A.Kd * (uint32_t)sizeof(XT) +
                                             L.g * (uint32_t)S::XBYTES
                                       : SK_OOB;
  sk_f32x4 acc[RT][1];
  S::template run_part<SV ? 4 : FEW_D>(acc, L, 0, (A.Kd + S::STEP - 1) / S::STEP, wave, FEW_W);
  sk_put<RT, 1>(red, acc);
  constexpr int OUT_TILES = GATE_UP ? RT / 2 : RT;
  for (int i = threadIdx.x; i < OUT_TILES * 64; i += 64 * FEW_W) {
    const int f = i >> 6, c = col0 + f * 16 + 4 * L.g;  // 64 threads to a tile: each its own lane's column
    if (j0 + (lane & 15) >= toks || c >= A.Nd) continue;  // Nd % 4 == 0: four columns exist or none
    const long long o = (long long)hr * A.Nd + c;
    const sk_f32x4 a = sk_get<FEW_W, RT, 1>(red, f, 0, lane);
    if constexpr (GATE_UP) {
      const sk_f32x4 b = sk_get<FEW_W, RT, 1>(red, f + RT / 2, 0, lane);
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = silu(a[q]) * b[q];
      if constexpr (sizeof(XT) == 4) {
        *reinterpret_cast<sk_f32x4*>(static_cast<float*>(A.out) + o) = sk_f32x4{v[0], v[1], v[2], v[3]};
      } else {
        // h is rounded to bf16, as the operand of the down projection's
        // matrix instructions (fp32 layers keep it in fp32)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.out) + o) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    } else {
      *reinterpret_cast<sk_f32x4*>(static_cast<float*>(A.out) + o) = a;
    }
  }
}

template <int WT, typename XT, bool GATE_UP, bool SV>
__global__ __launch_bounds__(64 * FEW_W) void k_few_product(FewArgs A) {
  __shared__ sk_f32x4 red[FEW_W * FEW_RT * 64];
  constexpr int COLS = GATE_UP ? FEW_RT * 8 : FEW_RT * 16;  // output columns of an item
  const int tiles = (A.Nd + COLS - 1) / COLS;
  const int e = blockIdx.x / tiles, col0 = (blockIdx.x % tiles) * COLS;
  const int lane = threadIdx.x & 63;
  // the shared experts come first: they have the most tokens
  int ex = A.Nr + e, toks = A.T;
  const int32_t* pairs = nullptr;
  int p = (lane & 15) << 16 | (A.K + e);
  if (e >= A.Ns) {
    // one memory latency for all four; what lies past the list is not used
    const int n = *A.lists.n;
    ex = A.lists.expert[e - A.Ns];
    toks = A.lists.tokens[e - A.Ns];
    pairs = A.lists.pair + (e - A.Ns) * FEW_T;
    p = pairs[lane & 15];
    if (e - A.Ns >= n) return;
  }
  // more than 16 tokens: the rows are read again, from a cache that has just
  // held them
  for (int j0 = 0; j0 < toks; j0 += 16) {
    if (j0) {
      p = pairs ? pairs[j0 + (lane & 15)] : p + (16 << 16);
      __syncthreads();  // red is read until here
    }
    few_item<WT, XT, GATE_UP, SV>(A, ex, toks, j0, p, col0, red);
  }
}

// --------------------------------------------------------------- combine --
template <typename RT, typename OT>
__global__ __launch_bounds__(128) void k_few_combine(const RT* resid, const float* __restrict__ y,
                                                     const float* __restrict__ gate, int d, int K, int Ns, OT* out) {
  const int t = blockIdx.x, c = (blockIdx.y * 128 + threadIdx.x) * 8;
  if (c >= d) return;
  float acc[8] = {}, v[8];
  if (resid) Vec8<RT>::load(resid + (long long)t * d + c, acc);
  const float* yt = y + (long long)t * (K + Ns) * d + c;
  for (int j = 0; j < Ns; ++j) {
    Vec8<float>::load(yt + (long long)(K + j) * d, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += v[i];
  }
  for (int k = 0; k < K; ++k) {
    const float g = gate[t * K + k];
    Vec8<float>::load(yt + (long long)k * d, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, v[i], acc[i]);
  }
  Vec8<OT>::store(out + (long long)t * d + c, acc);
}

template <int WT, typename XT, bool GATE_UP>
void launch_product(FewArgs a, int experts, hipStream_t st) {
  const int cols = GATE_UP ? FEW_RT * 8 : FEW_RT * 16;
  const dim3 grid(experts * ((a.Nd + cols - 1) / cols)), block(64 * FEW_W);
  if (WT == MOE_E2M1 && a.Kd % 128 == 0)
    hipLaunchKernelGGL((k_few_product<WT, XT, GATE_UP, WT == MOE_E2M1>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_few_product<WT, XT, GATE_UP, false>), grid, block, 0, st, a);
}

template <int WT, typename XT>
void launch_products(FewArgs up, FewArgs down, int experts, hipStream_t st) {
  launch_product<WT, XT, true>(up, experts, st);
  launch_product<WT, XT, false>(down, experts, st);
}

template <typename UT>
void launch_logits(const void* u, const float* e, int T, int d, int Nr, int parts, float* z, hipStream_t st) {
  const int step = Skinny<MOE_F32, UT, 1, 1>::STEP, steps = (d + step - 1) / step;
  const int per = (steps + parts - 1) / parts;
  const dim3 grid((Nr + 15) / 16, parts);
  if (T <= 16)
    hipLaunchKernelGGL((k_few_logits<UT, 1>), grid, dim3(64 * LOGIT_W), 0, st, static_cast<const UT*>(u), e, T, d, Nr,
                       per, z);
  else
    hipLaunchKernelGGL((k_few_logits<UT, 2>), grid, dim3(64 * LOGIT_W), 0, st, static_cast<const UT*>(u), e, T, d, Nr,
                       per, z);
}

template <typename RT, typename OT>
void launch_combine(const void* resid, const float* y, const float* gate, int T, int d, int K, int Ns, void* out,
                    hipStream_t st) {
  hipLaunchKernelGGL((k_few_combine<RT, OT>), dim3(T, (unsigned)ceil_div(d, 1024)), dim3(128), 0, st,
                     static_cast<const RT*>(resid), y, gate, d, K, Ns, static_cast<OT*>(out));
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
    launch_logits<float>(u, centroids, T, d, Nr, parts, w.z, st);
  else
    launch_logits<uint16_t>(u, centroids, T, d, Nr, parts, w.z, st);
  auto select = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, st, w.z, parts, bias, T, Nr, K, topk_idx, topk_gate, topk_score,
                       expert_load, w.lists);
  };
  if (Nr <= 64)
    select(k_few_select<1>);
  else if (Nr <= 256)
    select(k_few_select<4>);
  else
    select(k_few_select<16>);
  const FewArgs up{u, w13, w13_scale, w.h, w.lists, T, K, Nr, Ns, I, d};
  const FewArgs down{w.h, w2, w2_scale, w.y, w.lists, T, K, Nr, Ns, d, I};
  const int experts = Ns + (T * K < Nr ? T * K : Nr);
  switch (w_t) {
    case MOE_F32: launch_products<MOE_F32, float>(up, down, experts, st); break;
    case MOE_BF16: launch_products<MOE_BF16, uint16_t>(up, down, experts, st); break;
    case MOE_E4M3: launch_products<MOE_E4M3, uint16_t>(up, down, experts, st); break;
    default: launch_products<MOE_E2M1, uint16_t>(up, down, experts, st); break;
  }
  const bool rf = !resid || r_t == MOE_F32;
  if (out_t == MOE_F32) {
    if (rf) launch_combine<float, float>(resid, w.y, topk_gate, T, d, K, Ns, out, st);
    else launch_combine<uint16_t, float>(resid, w.y, topk_gate, T, d, K, Ns, out, st);
  } else {
    if (rf) launch_combine<float, uint16_t>(resid, w.y, topk_gate, T, d, K, Ns, out, st);
    else launch_combine<uint16_t, uint16_t>(resid, w.y, topk_gate, T, d, K, Ns, out, st);
  }
  return launch_status("moe_layer_few");
}

}  // namespace moe
