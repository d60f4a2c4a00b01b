// Root-mean-square norm in front of an expert layer, with the residual's
// addition and the 1x128 E4M3 tiles of its output, and its gradient.
//
//   r = x + resid,  c = (mean_j r_j^2 + eps)^(-1/2),  u = r c w
//   xhat = r c, g = du w:  dx = dr + c (g - xhat mean_j(g_j xhat_j)),
//                          dw_j = sum_t du_tj xhat_tj
// Both are bound by HBM: every operand is read once and every result written
// once, the row living in registers between the reduction and its use (a
// thread holds C chunks of 8 columns; TPR threads share a row).  Up to d = 8192
// nothing spills; of the forms beyond, most that have an fp32 operand do: the
// forward's for d > 16384 6 to 46 registers, the backward's 4 to 18, which
// live in scratch memory for that time.  A thread has read all it needs of a
// row before it writes any of it, so a result may lie on an operand of its own
// type.
// Measured, bf16: forward, 16384 rows of 7168, 173 us without tiles (5.4 TB/s
// of a half read, half written mix; a large copy reaches 4.8), 183 to 187 with
// them (5.7 TB/s), one row 2.8 us; backward 144 us (6.5 TB/s of three reads and
// a write), 8192 rows 93 us with k_norm_dw.  Few rows of wide d are the
// farthest from the bytes they need, since every block leaves a row of dw sums:
// 7168 columns, 256 rows 12.5 us for 3.1 of copying, 1024 rows 22 for 12, 2048
// rows 33 for 25.
#include "common.h"
#include "vec8.h"

namespace moe {

namespace {

constexpr int NORM_MAX_D = 1024 * 4 * 8;

// The longest rows leave no registers for w, nor for dr ahead of its use: both
// are then read where they are needed.
template <int TPR, int C>
constexpr bool norm_keeps_w() {
  return TPR * C <= 2048;
}

template <int TPR>
constexpr int norm_threads() {
  return TPR == 64 ? 256 : TPR;
}

// Sum of v over the TPR threads of a row.  `red` holds one value per wave for
// two rows in turn, so one barrier a row is enough: a wave that writes the
// next row's slot has passed the barrier after which the others read this
// row's, and the slot after that is two barriers away.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (&red)[2][16], int parity) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) red[parity][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[parity][0];
#pragma unroll
  for (int i = 1; i < TPR / 64; ++i) s += red[parity][i];
  return s;
}

__device__ __forceinline__ void load_w8(const void* w, bool bf16, int c, float (&v)[8]) {
  if (bf16)
    Vec8<uint16_t>::load(static_cast<const uint16_t*>(w) + c, v);
  else
    Vec8<float>::load(static_cast<const float*>(w) + c, v);
}

template <typename XT, typename RT, int TPR, int C>
__global__ __launch_bounds__(norm_threads<TPR>()) void k_rmsnorm(
    const XT* x, const RT* resid, const void* __restrict__ w, bool w_bf16, float eps, long long T, int d, RT* r_out,
    void* u, bool u_bf16, uint8_t* __restrict__ q,
    float* __restrict__ q_scale, float* __restrict__ rstd) {
  __shared__ float red[2][16];
  constexpr int RPB = norm_threads<TPR>() / TPR;  // rows a block works on at a time
  const int tid = threadIdx.x % TPR;
  constexpr bool KEEP = norm_keeps_w<TPR, C>();
  int col[C];
  bool live[C];
  float wv[KEEP ? C : 1][8];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    col[j] = (j * TPR + tid) * 8;
    live[j] = col[j] < d;
    if (KEEP && live[j]) load_w8(w, w_bf16, col[j], wv[j]);
  }
  int parity = 0;
  for (long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR; row < T; row += (long long)gridDim.x * RPB) {
    const long long o = row * d;
    float v[C][8];
    Raw8<XT> rx[C];
    Raw8<RT> rr[C];
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (live[j]) {
        rx[j].load(x + o + col[j]);
        if (resid) rr[j].load(resid + o + col[j]);
      }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (live[j]) {
        rx[j].get(v[j]);
        if (resid) {
          float t[8];
          rr[j].get(t);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] += t[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(v[j][i], v[j][i], s);
      }
    s = row_sum<TPR>(s, red, parity);
    parity ^= 1;
    const float c = 1.0f / sqrtf(s / (float)d + eps);
    if (rstd && tid == 0) rstd[row] = c;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      // 16 consecutive threads hold a 1x128 tile: all live or none (d % 128
      // == 0 where tiles are asked for)
      if (live[j]) {
        if (r_out) Vec8<RT>::store(r_out + o + col[j], v[j]);
        float y[8];
        float (&wj)[8] = wv[KEEP ? j : 0];
        if (!KEEP) load_w8(w, w_bf16, col[j], wj);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[j][i] * c * wj[i];
        if (u) {
          if (u_bf16)
            Vec8<uint16_t>::store(static_cast<uint16_t*>(u) + o + col[j], y);
          else
            Vec8<float>::store(static_cast<float*>(u) + o + col[j], y);
        }
        if (q) {
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
          for (int off = 1; off < 16; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
          const int k = pow2_scale_exp(amax);
          const float inv = exp2_int(-k);
          uint2 code;
          code.x = e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
          code.y = e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
          *reinterpret_cast<uint2*>(q + o + col[j]) = code;
          if ((tid & 15) == 0) q_scale[(o + col[j]) >> 7] = exp2_int(k);
        }
      }
    }
  }
}

// dx of every row, and this block's part of dw: each row group (the threads
// that share a row) adds rows group, group + groups, ... in registers, a
// block's groups are added through LDS and the blocks by k_norm_dw, all in the
// order of their number, so dw is bitwise reproducible.
template <typename GT, typename RT, int TPR, int C>
__global__ __launch_bounds__(norm_threads<TPR>()) void k_rmsnorm_bwd(
    const GT* du, const RT* r, const void* __restrict__ w, bool w_bf16, const float* __restrict__ rstd, const RT* dr,
    long long T, int d, RT* dx, float* __restrict__ part) {
  __shared__ float red[2][16];
  constexpr int RPB = norm_threads<TPR>() / TPR;
  const int tid = threadIdx.x % TPR;
  const long long group = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
  constexpr bool KEEP = norm_keeps_w<TPR, C>();
  int col[C];
  bool live[C];
  float wv[KEEP ? C : 1][8], dw[C][8];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    col[j] = (j * TPR + tid) * 8;
    live[j] = col[j] < d;
    if (KEEP && live[j]) load_w8(w, w_bf16, col[j], wv[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  int parity = 0;
  for (long long row = group; row < T; row += (long long)gridDim.x * RPB) {
    const long long o = row * d;
    Raw8<GT> rg[C];
    Raw8<RT> rr[C], rd[C];
    const float c = rstd[row];
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (live[j]) {
        rg[j].load(du + o + col[j]);
        rr[j].load(r + o + col[j]);
        if (KEEP && dr) rd[j].load(dr + o + col[j]);
      }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (live[j]) {
        float g[8], h[8];
        float (&wj)[8] = wv[KEEP ? j : 0];
        if (!KEEP) load_w8(w, w_bf16, col[j], wj);
        rg[j].get(g);
        rr[j].get(h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gx = g[i] * (h[i] * c);
          dw[j][i] += gx;
          s = fmaf(gx, wj[i], s);
        }
      }
    s = row_sum<TPR>(s, red, parity);
    parity ^= 1;
    const float m = s / (float)d;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (live[j]) {
        float g[8], h[8], out[8];
        float (&wj)[8] = wv[KEEP ? j : 0];
        if (!KEEP) load_w8(w, w_bf16, col[j], wj);
        rg[j].get(g);
        rr[j].get(h);
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = c * (g[i] * wj[i] - h[i] * c * m);
        if (dr) {
          float t[8];
          if (!KEEP) rd[j].load(dr + o + col[j]);
          rd[j].get(t);
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] += t[i];
        }
        Vec8<RT>::store(dx + o + col[j], out);
      }
  }
  if constexpr (RPB > 1) {
    __shared__ float sum[RPB - 1][C * TPR * 8];
    const int g = threadIdx.x / TPR;
    if (g > 0)
#pragma unroll
      for (int j = 0; j < C; ++j) Vec8<float>::store(&sum[g - 1][(j * TPR + tid) * 8], dw[j]);
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int o = 0; o < RPB - 1; ++o)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float t[8];
        Vec8<float>::load(&sum[o][(j * TPR + tid) * 8], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] += t[i];
      }
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (live[j]) Vec8<float>::store(part + (long long)blockIdx.x * d + col[j], dw[j]);
}

// dw[j] = sum over the blocks of part[., j].  A block owns 16 columns; its
// threads r of each column add parts r, r + 16, ... and one adds their sums.
// (64 columns and 16 waves to a block left 32 blocks at d = 2048: 38 us.)
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ part, int parts, int d,
                                                 float* __restrict__ dw) {
  __shared__ float red[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < d) {
    const float* p = part + (long long)r * d + col;
    int g = r;
    for (; g + 7 * 16 < parts; g += 8 * 16, p += 8 * 16 * (long long)d) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i * 16 * (long long)d];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; g < parts; g += 16, p += 16 * (long long)d) s += *p;
  }
  red[r][c] = s;
  __syncthreads();
  if (r == 0 && col < d) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][c];
    dw[col] = s;
  }
}

// Blocks of the backward: each leaves one row of dw sums, so few are wanted,
// and enough rows under way to cover the latency (bf16, 117M values: d = 264,
// 512 blocks 248 us, 1024 165, 2048 192; d = 1024, 512 blocks 141, 1024 147; d
// = 2048, 512 blocks 164, 1024 143, but 4096 rows with an fp32 stream 27 and
// 30; d = 7168, 256 blocks 102, 512 89, 768 97 for half as many values).
int norm_bwd_blocks(long long T, int d) {
  const long long need = d <= 1024 ? ceil_div(T, 4) : T, most = d <= 512 || (d > 1024 && d <= 2048 && T >= 16384) ? 1024 : 512;
  return (int)(need < most ? need : most);
}

bool is_fp(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16; }

// The fewest chunks a thread: every load of a row is then in flight at once
// and few registers let many rows be resident (16384 rows of 7168 bf16 with
// tiles: 1024 threads x 1 chunk 186 us, 512 x 2 194, 256 x 4 205; one row 2.9,
// 3.2, 4.0).  A block a row: rows taken in a loop of 2048 blocks 214 us.
template <typename XT, typename RT>
void launch_norm(const void* x, const void* resid, const void* w, bool w_bf16, float eps, long long T, int d,
                 void* r_out, void* u, bool u_bf16, uint8_t* q, float* q_scale, float* rstd, hipStream_t st) {
  auto go = [&](auto kernel, int threads, int rows) {
    // a launch has fewer than 2^32 threads; further rows in a loop
    const long long need = ceil_div(T, rows), most = 0xFFFFFFFFLL / threads;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(need < most ? need : most)), dim3(threads), 0, st,
                       static_cast<const XT*>(x), static_cast<const RT*>(resid), w, w_bf16, eps, T, d,
                       static_cast<RT*>(r_out), u, u_bf16, q, q_scale, rstd);
  };
  if (d <= 512)
    go(k_rmsnorm<XT, RT, 64, 1>, 256, 4);
  else if (d <= 2048)
    go(k_rmsnorm<XT, RT, 256, 1>, 256, 1);
  else if (d <= 4096)
    go(k_rmsnorm<XT, RT, 512, 1>, 512, 1);
  else if (d <= 8192)
    go(k_rmsnorm<XT, RT, 1024, 1>, 1024, 1);
  else if (d <= 16384)
    go(k_rmsnorm<XT, RT, 1024, 2>, 1024, 1);
  else
    go(k_rmsnorm<XT, RT, 1024, 4>, 1024, 1);
}

// The backward's blocks take rows in a loop, with dw in registers: more
// chunks a thread keep the rows' latencies apart (8192 rows of 7168 bf16: 256
// threads x 4 chunks 89 us, 1024 x 1 97, 512 x 2 98; 4096 rows of 2048, 256 x
// 1 24, 64 x 4 27).
template <typename GT, typename RT>
void launch_norm_bwd(const void* du, const void* r, const void* w, bool w_bf16, const float* rstd, const void* dr,
                     long long T, int d, void* dx, float* part, hipStream_t st) {
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3(norm_bwd_blocks(T, d)), dim3(threads), 0, st, static_cast<const GT*>(du),
                       static_cast<const RT*>(r), w, w_bf16, rstd, static_cast<const RT*>(dr), T, d,
                       static_cast<RT*>(dx), part);
  };
  if (d <= 512)
    go(k_rmsnorm_bwd<GT, RT, 64, 1>, 256);
  else if (d <= 1024)
    go(k_rmsnorm_bwd<GT, RT, 64, 2>, 256);
  else if (d <= 2048)
    go(k_rmsnorm_bwd<GT, RT, 256, 1>, 256);
  else if (d <= 8192)
    go(k_rmsnorm_bwd<GT, RT, 256, 4>, 256);
  else if (d <= 16384)
    go(k_rmsnorm_bwd<GT, RT, 1024, 2>, 1024);
  else
    go(k_rmsnorm_bwd<GT, RT, 1024, 4>, 1024);
}

bool norm_d_ok(int d) { return d >= 8 && d % 8 == 0 && d <= NORM_MAX_D; }

}  // namespace

moe_status rmsnorm(const void* x, moe_dtype x_t, const void* resid, moe_dtype r_t, const void* w, moe_dtype w_t,
                   float eps, long long T, int d, void* r_out, void* u, moe_dtype u_t, uint8_t* q, float* q_scale,
                   float* rstd, void* stream) {
  MOE_REQUIRE(is_fp(x_t) && is_fp(w_t), MOE_EINVAL, "x_t and w_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(!(resid || r_out) || is_fp(r_t), MOE_EINVAL, "r_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(!u || is_fp(u_t), MOE_EINVAL, "u_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(std::isfinite(eps) && eps >= 0.f, MOE_EINVAL, "eps must be finite and not negative");
  MOE_REQUIRE(T >= 0 && T < (1LL << 40) && d >= 8 && d % 8 == 0, MOE_EINVAL,
              "need T >= 0 and d a positive multiple of 8");
  MOE_REQUIRE(d <= NORM_MAX_D, MOE_EUNSUPPORTED, "d above 32768");
  MOE_REQUIRE((q == nullptr) == (q_scale == nullptr), MOE_EINVAL, "q and q_scale go together");
  MOE_REQUIRE(!q || d % 128 == 0, MOE_EINVAL, "E4M3 tiles need d % 128 == 0");
  MOE_REQUIRE(T == 0 || u || q, MOE_EINVAL, "u and q are both NULL");
  MOE_REQUIRE(T == 0 || (x && w), MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(x) && aligned16(resid) && aligned16(w) && aligned16(r_out) && aligned16(u) && aligned16(q),
              MOE_EINVAL, "x, resid, weight, r_out, u and q must be 16-byte aligned");
  if (T == 0) return MOE_OK;
  hipStream_t st = as_stream(stream);
  const bool rf = !(resid || r_out) || r_t == MOE_F32;
  auto go = [&](auto launch) {
    launch(x, resid, w, w_t == MOE_BF16, eps, T, d, r_out, u, u_t == MOE_BF16, q, q_scale, rstd, st);
  };
  if (x_t == MOE_F32) {
    if (rf) go(launch_norm<float, float>); else go(launch_norm<float, uint16_t>);
  } else {
    if (rf) go(launch_norm<uint16_t, float>); else go(launch_norm<uint16_t, uint16_t>);
  }
  return launch_status("moe_rmsnorm");
}

size_t rmsnorm_backward_workspace_bytes(long long T, int d) {
  if (T <= 0 || !norm_d_ok(d)) return 0;
  return (size_t)norm_bwd_blocks(T, d) * d * sizeof(float);
}

moe_status rmsnorm_backward(const void* du, moe_dtype du_t, const void* r, moe_dtype r_t, const void* w, moe_dtype w_t,
                            const float* rstd, const void* dr, long long T, int d, void* dx, float* dw, void* ws,
                            size_t ws_bytes, void* stream) {
  MOE_REQUIRE(is_fp(du_t) && is_fp(r_t) && is_fp(w_t), MOE_EINVAL, "du_t, r_t and w_t must be MOE_F32 or MOE_BF16");
  MOE_REQUIRE(T >= 0 && T < (1LL << 40) && d >= 8 && d % 8 == 0, MOE_EINVAL,
              "need T >= 0 and d a positive multiple of 8");
  MOE_REQUIRE(d <= NORM_MAX_D, MOE_EUNSUPPORTED, "d above 32768");
  MOE_REQUIRE(dw, MOE_EINVAL, "dw is NULL");
  MOE_REQUIRE(T == 0 || (du && r && w && rstd && dx), MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(du) && aligned16(r) && aligned16(w) && aligned16(dr) && aligned16(dx) && aligned16(ws),
              MOE_EINVAL, "du, r, weight, dr, dx and ws must be 16-byte aligned");
  MOE_REQUIRE(T == 0 || (ws && ws_bytes >= rmsnorm_backward_workspace_bytes(T, d)), MOE_EWORKSPACE,
              "workspace smaller than moe_rmsnorm_backward_workspace_bytes");
  hipStream_t st = as_stream(stream);
  float* part = static_cast<float*>(ws);
  if (T > 0) {
    auto go = [&](auto launch) { launch(du, r, w, w_t == MOE_BF16, rstd, dr, T, d, dx, part, st); };
    if (du_t == MOE_F32) {
      if (r_t == MOE_F32) go(launch_norm_bwd<float, float>); else go(launch_norm_bwd<float, uint16_t>);
    } else {
      if (r_t == MOE_F32) go(launch_norm_bwd<uint16_t, float>); else go(launch_norm_bwd<uint16_t, uint16_t>);
    }
  }
  // T == 0: no groups, dw = 0
  hipLaunchKernelGGL(k_norm_dw, dim3((d + 15) / 16), dim3(256), 0, st, part, T > 0 ? norm_bwd_blocks(T, d) : 0, d, dw);
  return launch_status("moe_rmsnorm_backward");
}

}  // namespace moe
