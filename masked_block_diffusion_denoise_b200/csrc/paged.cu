// The paged KV cache: block tables, free list and slot map from request
// lengths, and the write of new tokens' K and V into their slots.  (A finished
// block joins the cache of its sequence: course "Diffusion LLMs", section 14.)
#include <climits>

#include <cooperative_groups.h>

#include "kernels.h"

namespace dlm {

namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Resize.  With pages(n) = ceil(n / P), per sequence
//   need = max(0, pages(new) - pages(cur)), gone = max(0, pages(cur) - pages(new)),
//   tok = max(0, new - cur);
// three exclusive prefix sums over the batch (D, F, T) say everything else:
// the k-th new page of the batch is entry top-1-k of the stack, where the
// stack is the free list with the released pages pushed in reverse order, so
// k < F_total is released page k and the others come from the free list.
// Every thread can therefore compute any output by itself, and no output is
// read back: one launch, one cluster, no order of atomics.  Each CTA of the
// cluster scans the batch for itself (its sequences' state in shared memory)
// and then takes its share of the outputs; the cluster barrier between the
// two allows the outputs to overwrite the inputs.
// Bound by latency (a few hundred KB at most): one sequence that takes two pages
// 4.5 us a call in a graph, 256 requests of which the last do not get their
// pages 8.7, 48 prompts of up to 2000 tokens (48 thousand slots) 7.7.
// ---------------------------------------------------------------------------
constexpr int kResizeThreads = 1024;
constexpr int kResizeSeqs = kPagedMaxBatch;
constexpr int kRun = 4;   // consecutive slots of a thread: mostly one sequence and page

struct Scan3 {
  long long need, gone, tok;
};
__device__ __forceinline__ Scan3 operator+(const Scan3& a, const Scan3& b) {
  return Scan3{a.need + b.need, a.gone + b.gone, a.tok + b.tok};
}
__device__ __forceinline__ Scan3 shfl_up3(const Scan3& a, int d) {
  return Scan3{__shfl_up_sync(0xffffffffu, a.need, d), __shfl_up_sync(0xffffffffu, a.gone, d),
               __shfl_up_sync(0xffffffffu, a.tok, d)};
}

__device__ __forceinline__ Scan3 shfl3(const Scan3& a, int lane) {
  return Scan3{__shfl_sync(0xffffffffu, a.need, lane), __shfl_sync(0xffffffffu, a.gone, lane),
               __shfl_sync(0xffffffffu, a.tok, lane)};
}

// largest i in [0, n) with first[i] <= x, for ascending first, first[0] <= x
__device__ __forceinline__ int find_last(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kResizeThreads, 1) resize_kernel(const PagedResize a) {
  extern __shared__ int sm[];
  int* s_cur = sm;               // [B] length now
  int* s_new = s_cur + a.B;      // [B] length wanted
  int* s_need = s_new + a.B;     // [B] D: new pages before this sequence's
  int* s_gone = s_need + a.B;    // [B] F: released pages before this sequence's
  int* s_tok = s_gone + a.B;     // [B] T: new tokens before this sequence's, capped at max_new
  int* s_ok = s_tok + a.B;       // [B] served
  __shared__ Scan3 warp_sum[32];
  __shared__ unsigned long long s_taken;   // pages taken

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, n_ranks = gridDim.x;
  const int sh = a.page_shift;
  const long long page_mask = (1ll << sh) - 1;
  pdl_wait_then_release();
  const int n_free = *a.n_free_in;
  auto pages = [&](int n) { return (int)(((long long)n + page_mask) >> sh); };

  // this thread's consecutive sequences
  const int per = (a.B + kResizeThreads - 1) / kResizeThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto change = [&](int cur, int want) {
    Scan3 c{0, 0, 0};
    if (cur < 0 || want < 0) return c;
    const int pc = pages(cur), pn = pages(want);
    if (pn <= a.W && pc <= a.W) {
      c.need = max(0, pn - pc);
      c.gone = max(0, pc - pn);
    }
    c.tok = max(0, want - cur);
    return c;
  };
  Scan3 mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int cur = a.cur[b], want = a.want[b];
    s_cur[b] = cur;
    s_new[b] = want;
    mine = mine + change(cur, want);
  }
  auto warp_scan = [&](Scan3 x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Scan3 o = shfl_up3(x, d);
      if (lane >= d) x = x + o;
    }
    return x;
  };
  const Scan3 incl = warp_scan(mine);
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) s_taken = 0;
  __syncthreads();
  // every warp scans the warps' sums
  static_assert(kResizeThreads == 1024, "a lane per warp");
  const Scan3 sums = warp_scan(warp_sum[lane]);
  const Scan3 all = shfl3(sums, 31), upto = shfl3(sums, warp);
  // before this thread's sequences
  const Scan3 own = warp_sum[warp];
  Scan3 at = Scan3{upto.need - own.need + incl.need - mine.need,
                   upto.gone - own.gone + incl.gone - mine.gone,
                   upto.tok - own.tok + incl.tok - mine.tok};
  // a broken stack: nothing changes
  const bool broken = n_free < 0 || n_free > a.n_pages || n_free + all.gone > a.n_pages;
  const long long have = broken ? 0 : n_free + all.gone;
  long long taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int cur = s_cur[b], want = s_new[b];
    const Scan3 c = change(cur, want);
    const bool fits = cur >= 0 && want >= 0 && pages(want) <= a.W && pages(cur) <= a.W;
    const bool ok = !broken && fits && (c.need == 0 || at.need + c.need <= have) &&
                    (c.tok == 0 || at.tok + c.tok <= a.max_new);
    s_ok[b] = ok;
    s_need[b] = (int)min(at.need, (long long)INT_MAX);
    s_gone[b] = (int)min(at.gone, (long long)INT_MAX);
    s_tok[b] = (int)min(at.tok, (long long)a.max_new);
    if (ok) taken += c.need;
    at = at + c;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) taken += __shfl_xor_sync(0xffffffffu, taken, d);
  // whole numbers: the order of the additions does not matter
  if (lane == 0 && taken > 0)
    atomicAdd(&s_taken, (unsigned long long)taken);
  __syncthreads();
  // every CTA has read the lengths and the stack's height
  if (n_ranks > 1) cg::this_cluster().sync();

  const int F = broken ? 0 : (int)all.gone;
  const int K = (int)s_taken;
  const int n_tok = (int)min(all.tok, (long long)a.max_new);
  // page id j of the released ones, and the k-th popped one
  auto checked = [&](int page) {
    if (page < 0 || page >= a.n_pages) raise_error(a.err, DLM_EBOUNDS);
    return page;
  };
  auto released = [&](int j) {
    const int b = find_last(s_gone, a.B, j);
    return checked(a.table[(size_t)b * a.W + pages(s_new[b]) + (j - s_gone[b])]);
  };
  auto popped = [&](int k) {
    return k < F ? released(k) : checked(a.free_pages[n_free + F - 1 - k]);
  };
  // outputs, as one list of tasks over the cluster's threads (neighbouring warps'
  // go to different CTAs), so that their chains of loads run side by side
  const int first = (warp * n_ranks + rank) * 32 + lane, step = n_ranks * kResizeThreads;
  if (first == 0) {
    if (broken) raise_error(a.err, DLM_EBOUNDS);
    *a.n_free_out = broken ? n_free : n_free + F - K;
    a.cu[0] = 0;
  }
  const int kept = max(0, F - K);                      // released pages that stay on the stack
  const int runs = (a.max_new + kRun - 1) / kRun;      // of the slot map
  const long long tasks = (long long)a.B + K + kept + runs;
  for (long long x = first; x < tasks; x += step) {
    long long y = x;
    if (y < runs) {
      // a slot per new token; a run's sequence and page are looked up when they change
      const int t0 = (int)y * kRun;
      int64_t slot[kRun];
      int b = -1, end = t0, col = -1, cur = 0, tb = 0, page_b = 0;
      bool ok = false;
      int64_t base = -1;
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        const int t = t0 + u;
        slot[u] = -1;
        if (t >= n_tok) continue;
        if (t >= end) {
          b = find_last(s_tok, a.B, t);
          end = b + 1 < a.B ? s_tok[b + 1] : n_tok;
          ok = s_ok[b] != 0;
          cur = s_cur[b];
          tb = s_tok[b];
          page_b = s_need[b] - pages(cur);
          col = -1;
        }
        if (!ok) continue;
        const int pos = cur + (t - tb);
        if (pos >> sh != col) {
          col = pos >> sh;
          const int page = col < pages(cur) ? checked(a.table[(size_t)b * a.W + col])
                                            : popped(page_b + col);
          base = page >= 0 && page < a.n_pages ? (int64_t)page << sh : -1;
        }
        if (base >= 0) slot[u] = base + (pos & (int)page_mask);
      }
      if (t0 + kRun <= a.max_new && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
        longlong2* dst = reinterpret_cast<longlong2*>(a.slots + t0);
        dst[0] = make_longlong2(slot[0], slot[1]);
        dst[1] = make_longlong2(slot[2], slot[3]);
      } else {
#pragma unroll
        for (int u = 0; u < kRun; ++u)
          if (t0 + u < a.max_new) a.slots[t0 + u] = slot[u];
      }
      continue;
    }
    y -= runs;
    if (y < K) {
      // a new page into its table (served sequences that need pages are the first
      // of those that need any, so page k's owner is found in D)
      const int k = (int)y, b = find_last(s_need, a.B, k);
      a.table[(size_t)b * a.W + pages(s_cur[b]) + (k - s_need[b])] = popped(k);
      continue;
    }
    y -= K;
    if (y < kept) {
      // position n_free + y of the stack
      a.free_pages[n_free + (int)y] = released(F - 1 - (int)y);
      continue;
    }
    const int b = (int)(y - kept);
    a.out_lens[b] = s_ok[b] ? s_new[b] : s_cur[b];
    a.cu[b + 1] = b + 1 < a.B ? s_tok[b + 1] : n_tok;
  }
}

// ---------------------------------------------------------------------------
// K/V rows into their slots: a copy in 16-byte pieces, bound by HBM (read once,
// written once).  Neighbouring threads take neighbouring pieces of a row, K's
// and V's loaded before either is stored, so that both are under way at once: 250 MB
// (30512 tokens, 8 heads x 128 in bf16) in 40.6 us, 6.16 TB/s; stored one after the
// other 44.9.  A block takes the rows that give each thread a piece (1024 tokens:
// 2.4 us a call in a graph; two pieces a thread 2.6 and 40.5, four 3.2 and 41.7).
// ---------------------------------------------------------------------------
constexpr int kWriteThreads = 256;
// (No __restrict__: the kernel before, which may write these, can still run
// when this one starts, so they are not read-only for its whole life.)
__global__ void __launch_bounds__(kWriteThreads)
    kv_write_kernel(const PagedKV c, const uint8_t* k, const uint8_t* v, int64_t k_stride,
                    int64_t v_stride, const int64_t* slots, int n, int tokens, int* err) {
  pdl_wait_then_release();
  const uint32_t head_chunks = (uint32_t)(c.Dh * c.esize / 16);
  const uint32_t row_chunks = (uint32_t)c.Hkv * head_chunks;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const uint32_t pieces = (uint32_t)min((int64_t)tokens, n - t0) * row_chunks;
  for (uint32_t i = threadIdx.x; i < pieces; i += kWriteThreads) {   // (long rows: more)
    const int64_t t = t0 + i / row_chunks;
    const uint32_t j = i % row_chunks;
    const int64_t slot = slots[t];
    if (slot < 0) continue;
    const int64_t page = slot >> c.page_shift;
    if (page >= c.n_pages) {
      raise_error(err, DLM_EBOUNDS);
      continue;
    }
    const int off = (int)(slot & ((1 << c.page_shift) - 1));
    const uint32_t head = j / head_chunks, part = j % head_chunks;
    const size_t dst = ((((size_t)page * c.Hkv + head) << c.page_shift) + off) * head_chunks + part;
    const uint4 a = *reinterpret_cast<const uint4*>(k + t * k_stride + j * 16);
    const uint4 b = *reinterpret_cast<const uint4*>(v + t * v_stride + j * 16);
    reinterpret_cast<uint4*>(c.k)[dst] = a;
    reinterpret_cast<uint4*>(c.v)[dst] = b;
  }
}

}  // namespace

cudaError_t paged_resize(const PagedResize& a, cudaStream_t st) {
  const int smem = 6 * a.B * (int)sizeof(int);
  static_assert(6 * kResizeSeqs * sizeof(int) <= 227 * 1024 - 2048, "batch exceeds shared memory");
  static DeviceOnce once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                6 * kResizeSeqs * (int)sizeof(int));
  });
  if (e != cudaSuccess) return e;
  // One CTA up to a run of slots a thread, then a cluster of up to 8: a CTA more
  // repeats the scan but shares the slots' stores.
  int ranks = 1;
  while (ranks < 8 && (long long)ranks * kRun * kResizeThreads < a.max_new) ranks *= 2;
  if (ranks == 1) return launch_pdl(resize_kernel, dim3(1), dim3(kResizeThreads), smem, st, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kResizeThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, resize_kernel, a);
}

cudaError_t paged_kv_write(const PagedKV& c, const void* k, const void* v, int64_t k_stride,
                           int64_t v_stride, const int64_t* slots, int n, int* err,
                           cudaStream_t st) {
  // rows of a block: a piece per thread, or one row of any length
  const int row_chunks = c.Hkv * (c.Dh * c.esize / 16);
  const int tokens = max(1, kWriteThreads / row_chunks);
  return launch_pdl(kv_write_kernel, dim3((unsigned)(((int64_t)n + tokens - 1) / tokens)),
                    dim3(kWriteThreads), 0, st, c, (const uint8_t*)k, (const uint8_t*)v,
                    k_stride * c.esize, v_stride * c.esize, slots, n, tokens, err);
}

}  // namespace dlm
