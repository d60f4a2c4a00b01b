// The paged latent cache: which pages a request's new tokens take, where each
// token lies, pages given back, and the rows written there.
//
//   have_b = ceil(len_b / P), want_b = ceil((len_b + new_b) / P)
//   page of token j of request b: table[b, j / P]; slot P page + j % P
// Requests are served in order; the i-th page that a step takes is the i-th
// from the top of the stack of free pages.  A request that does not fit gets
// no page and no slot.
//
// All latency: a block scans the requests' pages (64 requests of one token: 5.3
// us, of which an empty launch takes 2), a wide launch places the tokens of large
// steps (509 prompts, 260 thousand tokens: 5.2 + 5.6 us).
#include "mla.h"

namespace moe {

namespace {

constexpr int PG_THREADS = 1024;
// Tokens and requests up to which one block does it all: 4096 tokens 9.6 us a call
// where a second launch makes it 12.1, 8192 13.0 where that makes it 12.0.
constexpr int PG_ONE_BLOCK = 4096;
constexpr int PG_MAX_B = 8192;

struct PagePlan {  // of a request
  int cu;          // tokens of the requests before it
  int old;         // its length before the step
  int rank;        // pages that the step takes before its first, or -1 if it is not served
};

// Exclusive sum of v over the block's threads, and the total.
__device__ __forceinline__ long long block_scan(long long v, long long* wave_sum, long long& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long s = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long long t = __shfl_up(s, off, 64);
    if (lane >= off) s += t;
  }
  __syncthreads();
  if (lane == 63) wave_sum[wave] = s;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < PG_THREADS / 64; ++i) {
    if (i < wave) before += wave_sum[i];
    total += wave_sum[i];
  }
  return before + s - v;
}

struct PageArgs {
  const int32_t *seq_len, *new_len;
  int B, P;
  int32_t* table;
  int W;
  const int32_t* free_pages;
  int F;
  const int32_t* n_free;
  int32_t *seq_len_out, *n_free_out, *n_failed, *cu_new, *slot, *position;
  int N;
};

// One token: its request by bisection, its slot, and its page's entry in the
// table if it is the page's first.
__device__ __forceinline__ void page_token(const PageArgs& a, const PagePlan* plan, int total, int n_free, int t) {
  int slot = -1, pos = -1;
  if (t < total) {
    int lo = 0, hi = a.B;  // plan[lo].cu <= t < plan[hi].cu
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (plan[mid].cu <= t)
        lo = mid;
      else
        hi = mid;
    }
    const PagePlan q = plan[lo];
    pos = q.old + (t - q.cu);
    if (q.rank >= 0) {
      const int have = (int)(((uint32_t)q.old + a.P - 1u) / a.P), page_no = pos / a.P, at = pos - page_no * a.P;
      int32_t* entry = a.table + (long long)lo * a.W + page_no;
      int page;
      if (page_no < have) {
        page = *entry;
      } else {
        page = a.free_pages[n_free - 1 - (q.rank + page_no - have)];
        if (at == 0) *entry = page;
      }
      slot = page * a.P + at;
    }
  }
  a.slot[t] = slot;
  a.position[t] = pos;
}

// One block: the plan of every request (kept in LDS, or left in `plan_out`
// for k_pages_tokens), the totals, and with ALL every token.  All that the
// step replaces is read before the barrier that precedes its writing, so the
// outputs may be the inputs.
template <bool ALL>
__global__ __launch_bounds__(PG_THREADS) void k_pages_extend(PageArgs a, PagePlan* plan_out) {
  extern __shared__ PagePlan lds_plan[];
  __shared__ long long wave_sum[PG_THREADS / 64];
  PagePlan* plan = ALL ? lds_plan : plan_out + 1;  // plan_out[0] holds the totals
  const int per = (a.B + PG_THREADS - 1) / PG_THREADS, b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
  const int n_free = max(0, min(*a.n_free, a.F));
  // a thread's first request stays in registers: up to 1024 are read once
  const int old0 = b0 < b1 ? max(0, a.seq_len[b0]) : 0, add0 = b0 < b1 ? max(0, a.new_len[b0]) : 0;
  auto read = [&](int b, int& old, int& add) {
    old = b == b0 ? old0 : max(0, a.seq_len[b]);
    add = b == b0 ? add0 : max(0, a.new_len[b]);
  };
  auto need = [&](int old, int add, long long cu) -> int {  // pages, or -1 for a request that can't be served
    const long long len = (long long)old + add;
    if (add == 0) return 0;
    if (len > 0x7FFFFFFF || cu + add > a.N) return -1;
    const int have = (int)(((uint32_t)old + a.P - 1u) / a.P), want = (int)(((uint32_t)len + a.P - 1u) / a.P);
    return want <= a.W ? want - have : -1;
  };
  long long tok = 0, pages = 0, total_tok, total_pages;
  for (int b = b0; b < b1; ++b) {
    int old, add;
    read(b, old, add);
    tok += add;
  }
  const long long cu0 = block_scan(tok, wave_sum, total_tok);
  long long cu = cu0;
  for (int b = b0; b < b1; ++b) {
    int old, add;
    read(b, old, add);
    pages += max(0, need(old, add, cu));
    cu += add;
  }
  const long long first = block_scan(pages, wave_sum, total_pages);
  long long rank = first, given = 0;  // pages given, and in the low half the requests not served
  cu = cu0;
  for (int b = b0; b < b1; ++b) {
    int old, add;
    read(b, old, add);
    const int n = need(old, add, cu);
    const bool served = n == 0 || (n > 0 && rank + n <= n_free);
    plan[b] = {(int)min(cu, 0x7FFFFFFFLL), old, served ? (int)min(rank, 0x7FFFFFFFLL) : -1};
    given += ((long long)(served ? n : 0) << 32) + !served;
    rank += max(0, n);
    cu += add;
  }
  long long sums;
  block_scan(given, wave_sum, sums);
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    int old, add;
    read(b, old, add);
    a.cu_new[b] = plan[b].cu;
    a.seq_len_out[b] = plan[b].old + (plan[b].rank >= 0 ? add : 0);
  }
  const int total = (int)min(total_tok, 0x7FFFFFFFLL);
  if (threadIdx.x == 0) {
    a.cu_new[a.B] = total;
    *a.n_free_out = n_free - (int)(sums >> 32);
    *a.n_failed = (int)sums;
    if (!ALL) plan_out[0] = {total, n_free, 0};
  }
  if (ALL)
    for (int t = threadIdx.x; t < a.N; t += PG_THREADS) page_token(a, plan, total, n_free, t);
}

__global__ __launch_bounds__(256) void k_pages_tokens(PageArgs a, const PagePlan* plan) {
  const int total = plan[0].cu, n_free = plan[0].old;
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  if (t < a.N) page_token(a, plan + 1, total, n_free, (int)t);
}

// One block: pages of the requests marked in `done` onto the stack, in the
// order of requests and pages; their lengths to zero.  64 requests of 64 pages: 4.6
// us; 509 of 32: 15.4, a request to a wave 32 times in turn.
__global__ __launch_bounds__(PG_THREADS) void k_pages_release(const int32_t* __restrict__ done, int32_t* seq_len, int B,
                                                              int P, const int32_t* __restrict__ table, int W,
                                                              int32_t* free_pages, int F, int32_t* n_free) {
  extern __shared__ int first[];  // [B] place of a request's first page on the stack, or -1
  __shared__ long long wave_sum[PG_THREADS / 64];
  const int per = (B + PG_THREADS - 1) / PG_THREADS, b0 = threadIdx.x * per, b1 = min(B, b0 + per);
  const int top = max(0, min(*n_free, F));
  auto count = [&](int b) {
    return done[b] ? (int)min(((long long)max(0, seq_len[b]) + P - 1) / P, (long long)W) : 0;
  };
  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += count(b);
  long long at = top + block_scan(mine, wave_sum, total);
  for (int b = b0; b < b1; ++b) {
    const int n = count(b);
    first[b] = n ? (int)min(at, (long long)F) : -1;
    at += n;
  }
  __syncthreads();
  for (int b = threadIdx.x >> 6; b < B; b += PG_THREADS / 64) {
    if (first[b] < 0) continue;
    const int n = count(b);
    for (int i = threadIdx.x & 63; i < n && (long long)first[b] + i < F; i += 64)
      free_pages[first[b] + i] = table[(long long)b * W + i];
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b)
    if (done[b]) seq_len[b] = 0;
  if (threadIdx.x == 0) *n_free = (int)min((long long)F, top + total);
}

// A thread copies 16 bytes; a token without a slot, or with one outside the
// cache, is not written.  32768 tokens of 576: 13.8 us, 5.5 TB/s of bytes read and
// written; 8 tokens 2.3 us, the launch.
__global__ __launch_bounds__(256) void k_cache_write(const uint16_t* __restrict__ c, long long ldc,
                                                     const uint16_t* __restrict__ r, long long ldr,
                                                     const int32_t* __restrict__ slot, long long T, int dc, int dr,
                                                     uint16_t* __restrict__ cache, long long n_slots) {
  const int cc = dc / 8, per = cc + dr / 8;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < T * per; i += (long long)gridDim.x * 256) {
    const long long t = i / per;
    const int k = (int)(i - t * per);
    const long long at = slot[t];
    if (at < 0 || at >= n_slots) continue;
    const uint16_t* from = k < cc ? c + t * ldc + k * 8 : r + t * ldr + (k - cc) * 8;
    *reinterpret_cast<u32x4_t*>(cache + at * (dc + dr) + k * 8) = *reinterpret_cast<const u32x4_t*>(from);
  }
}

}  // namespace

size_t pages_workspace_bytes(int B) { return B < 1 || B > PG_MAX_B ? 0 : (size_t)(B + 1) * sizeof(PagePlan); }

moe_status pages_extend(const int32_t* seq_len, const int32_t* new_len, int B, int page_size, int32_t* table, int W,
                        const int32_t* free_pages, int F, const int32_t* n_free, int32_t* seq_len_out,
                        int32_t* n_free_out, int32_t* n_failed, int32_t* cu_new, int32_t* slot, int32_t* position,
                        int N, void* ws, size_t ws_bytes, void* stream) {
  MOE_REQUIRE(B >= 0 && page_size >= 1 && W >= 1 && F >= 0 && N >= 0, MOE_EINVAL,
              "need B, F, N >= 0 and page_size, W >= 1");
  MOE_REQUIRE(B <= PG_MAX_B, MOE_EUNSUPPORTED, "more requests than MLA_MAX_REQUESTS");
  MOE_REQUIRE(n_free && n_free_out && n_failed && cu_new && (N == 0 || (slot && position)), MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(B == 0 || (seq_len && new_len && table && seq_len_out && (F == 0 || free_pages)), MOE_EINVAL,
              "NULL pointer");
  const bool one = B == 0 || (N <= PG_ONE_BLOCK && B <= PG_ONE_BLOCK);
  MOE_REQUIRE(one || (ws && ws_bytes >= pages_workspace_bytes(B)), MOE_EWORKSPACE,
              "workspace smaller than mla_pages_workspace_bytes");
  MOE_REQUIRE(aligned4(ws), MOE_EINVAL, "ws must be 4-byte aligned");
  const PageArgs a{seq_len,     new_len,    B,        page_size, table, W,        free_pages, F, n_free,
                   seq_len_out, n_free_out, n_failed, cu_new,    slot,  position, N};
  hipStream_t st = as_stream(stream);
  if (one) {
    hipLaunchKernelGGL(k_pages_extend<true>, dim3(1), dim3(PG_THREADS), sizeof(PagePlan) * (B + 1), st, a, nullptr);
  } else {
    PagePlan* plan = static_cast<PagePlan*>(ws);
    hipLaunchKernelGGL(k_pages_extend<false>, dim3(1), dim3(PG_THREADS), 0, st, a, plan);
    hipLaunchKernelGGL(k_pages_tokens, dim3((unsigned)ceil_div(N, 256)), dim3(256), 0, st, a, plan);
  }
  return launch_status("mla_pages_extend");
}

moe_status pages_release(const int32_t* done, int32_t* seq_len, int B, int page_size, const int32_t* table, int W,
                         int32_t* free_pages, int F, int32_t* n_free, void* stream) {
  MOE_REQUIRE(B >= 0 && page_size >= 1 && W >= 1 && F >= 0, MOE_EINVAL, "need B, F >= 0 and page_size, W >= 1");
  MOE_REQUIRE(B <= PG_MAX_B, MOE_EUNSUPPORTED, "more requests than MLA_MAX_REQUESTS");
  MOE_REQUIRE(B == 0 || (done && seq_len && table && n_free && (F == 0 || free_pages)), MOE_EINVAL, "NULL pointer");
  if (B == 0) return MOE_OK;
  hipLaunchKernelGGL(k_pages_release, dim3(1), dim3(PG_THREADS), sizeof(int) * B, as_stream(stream), done, seq_len, B,
                     page_size, table, W, free_pages, F, n_free);
  return launch_status("mla_pages_release");
}

moe_status cache_write(const void* c, long long ldc, const void* r, long long ldr, const int32_t* slot, long long T,
                       int dc, int dr, void* cache, long long n_slots, void* stream) {
  MOE_REQUIRE(T >= 0 && T < (1LL << 31) && n_slots >= 0 && n_slots < (1LL << 31), MOE_EINVAL,
              "need 0 <= T, n_slots < 2^31");
  MOE_REQUIRE(dc >= 8 && dc % 8 == 0 && dr >= 8 && dr % 8 == 0, MOE_EINVAL,
              "dc and dr must be positive multiples of 8");
  MOE_REQUIRE(mla_dc_ok(dc) && dr <= MLA_MAX_DR, MOE_EUNSUPPORTED, "dc above 512 or dr above 64");
  MOE_REQUIRE(ldc >= dc && ldr >= dr && ldc % 8 == 0 && ldr % 8 == 0 && ldc < (1LL << 32) && ldr < (1LL << 32),
              MOE_EINVAL, "row strides must be multiples of 8 that hold a row");
  MOE_REQUIRE(T == 0 || (c && r && slot && (cache || n_slots == 0)), MOE_EINVAL, "NULL pointer");
  MOE_REQUIRE(aligned16(c) && aligned16(r) && aligned16(cache), MOE_EINVAL,
              "latent, k_rope and cache must be 16-byte aligned");
  if (T == 0 || n_slots == 0) return MOE_OK;
  const long long need = ceil_div(T * ((dc + dr) / 8), 256);
  hipLaunchKernelGGL(k_cache_write, dim3((unsigned)(need < 8192 ? need : 8192)), dim3(256), 0, as_stream(stream),
                     static_cast<const uint16_t*>(c), ldc, static_cast<const uint16_t*>(r), ldr, slot, T, dc, dr,
                     static_cast<uint16_t*>(cache), n_slots);
  return launch_status("mla_cache_write");
}

}  // namespace moe
