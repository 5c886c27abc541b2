// The paged KV cache: block tables, free list and slot map from request
// lengths, and the write of new tokens' K and V into their slots.  (A finished
// block joins the cache of its sequence: course "Diffusion LLMs", section 14.)
#include <algorithm>
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
// cluster scans the batch for itself (its sequences' state in shared memory),
// looks at every page id that the call uses, and then takes its share of the
// outputs; the cluster barrier between the two allows the outputs to overwrite
// the inputs.
// Bound by latency (a few hundred KB at most): one sequence that takes two pages
// 4.8 us a call in a graph, 256 requests of which the last do not get their
// pages 8.1, 48 prompts of up to 2000 tokens (48 thousand slots) 8.6 (4.5, 8.7 and
// 7.7 when the ids were not looked at before the outputs).
// ---------------------------------------------------------------------------
constexpr int kResizeThreads = 1024;
constexpr int kResizeSeqs = kPagedMaxBatch;
// Page ids kept in shared memory; beyond those (pools where a call releases or takes
// more) an id is looked up again where it is used.  (Looked up again everywhere, by
// searches in the scan: 10.2 us for the 256 requests, 8.7 for the prompts.)
constexpr int kResizeIds = 8192;
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

// four bytes into shared memory, without a register in between
__device__ __forceinline__ void copy4(int* dst, const int32_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kResizeThreads, 1) resize_kernel(const PagedResize a) {
  extern __shared__ int sm[];
  int* s_cur = sm;               // [B] length now
  int* s_new = s_cur + a.B;      // [B] length wanted
  int* s_need = s_new + a.B;     // [B] D: new pages before this sequence's
  int* s_gone = s_need + a.B;    // [B] F: released pages before this sequence's
  int* s_tok = s_gone + a.B;     // [B] T: new tokens before this sequence's, capped at max_new
  // [B] served sequences: the page they have begun (0 if none); -1 for refused ones
  int* s_begun = s_tok + a.B;
  int* s_ids = s_begun + a.B;       // [n_ids] the first popped or released page ids
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
  // the page that a growing sequence has begun; of the thread's last one it is loaded
  // here, so that it comes during the scan
  auto begun = [&](int b, int cur, int want) {
    return cur > 0 && want > cur && (cur & page_mask) != 0 && (cur >> sh) < a.W
               ? a.table[(size_t)b * a.W + (cur >> sh)]
               : 0;
  };
  int begun_last = 0;
  for (int b = b0; b < b1; ++b) {
    const int cur = a.cur[b], want = a.want[b];
    s_cur[b] = cur;
    s_new[b] = want;
    if (b == b1 - 1) begun_last = begun(b, cur, want);
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
  auto valid = [&](int page) { return page >= 0 && page < a.n_pages; };
  long long taken = 0;
  bool bad = false;   // a page id outside the cache among those that the call uses
  for (int b = b0; b < b1; ++b) {
    const int cur = s_cur[b], want = s_new[b];
    const Scan3 c = change(cur, want);
    const bool fits = cur >= 0 && want >= 0 && pages(want) <= a.W && pages(cur) <= a.W;
    const bool ok = !broken && fits && (c.need == 0 || at.need + c.need <= have) &&
                    (c.tok == 0 || at.tok + c.tok <= a.max_new);
    s_need[b] = (int)min(at.need, (long long)INT_MAX);
    s_gone[b] = (int)min(at.gone, (long long)INT_MAX);
    s_tok[b] = (int)min(at.tok, (long long)a.max_new);
    if (ok) taken += c.need;
    const int page = b == b1 - 1 ? begun_last : begun(b, cur, want);
    bad |= ok && !valid(page);
    s_begun[b] = ok ? max(page, 0) : -1;
    at = at + c;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) taken += __shfl_xor_sync(0xffffffffu, taken, d);
  // whole numbers: the order of the additions does not matter
  if (lane == 0 && taken > 0)
    atomicAdd(&s_taken, (unsigned long long)taken);
  __syncthreads();
  int F = broken ? 0 : (int)all.gone;
  int K = (int)s_taken;
  const int n_tok = (int)min(all.tok, (long long)a.max_new);
  // Page ids: number k is the k-th popped one, below F also the k-th released one.  All
  // that the call uses are looked at before any output: one outside the cache would go
  // on to the stack or to another sequence, so the call changes nothing, as with a
  // broken stack.  Every CTA copies them to shared memory (the first n_ids), where the
  // outputs find them: a warp the released ones of its sequences, all copies under way
  // at once.
  const int n_ids = min(a.n_pages, kResizeIds), used = max(F, K);
  auto first_of = [&](int b) { return a.table + (size_t)b * a.W + pages(s_new[b]); };
  auto lookup = [&](int k) {
    if (k >= F) return a.free_pages[n_free + F - 1 - k];
    const int b = find_last(s_gone, a.B, k);
    return first_of(b)[k - s_gone[b]];
  };
  for (int b = lane * 32 + warp; F > 0 && b - lane * 32 < a.B; b += kResizeThreads) {
    const int from = b < a.B ? s_gone[b] : 0;
    const int n = b < a.B ? (b + 1 < a.B ? s_gone[b + 1] : F) - from : 0;
    for (uint32_t some = __ballot_sync(0xffffffffu, n > 0); some != 0; some &= some - 1) {
      const int l = __ffs(some) - 1;
      const int32_t* src = first_of(__shfl_sync(0xffffffffu, b, l));
      const int to = __shfl_sync(0xffffffffu, from, l);
      const int end = min(__shfl_sync(0xffffffffu, n, l), n_ids - to);
      for (int c = lane; c < end; c += 32) copy4(s_ids + to + c, src + c);
    }
  }
  for (int k = F + tid; k < min(K, n_ids); k += kResizeThreads)
    copy4(s_ids + k, a.free_pages + (n_free + F - 1 - k));
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  for (int k = tid; k < min(used, n_ids); k += kResizeThreads) bad |= !valid(s_ids[k]);
  for (int k = n_ids + tid; k < used; k += kResizeThreads) bad |= !valid(lookup(k));
  auto taken_page = [&](int k) { return k < n_ids ? s_ids[k] : lookup(k); };
  const bool stop = __syncthreads_or(bad) || broken;
  if (stop) F = K = 0;
  // every CTA has read the lengths, the tables and the stack
  if (n_ranks > 1) cg::this_cluster().sync();
  // outputs, as one list of tasks over the cluster's threads (neighbouring warps'
  // go to different CTAs), so that their chains of loads run side by side
  const int first = (warp * n_ranks + rank) * 32 + lane, step = n_ranks * kResizeThreads;
  if (first == 0) {
    if (stop) raise_error(a.err, DLM_EBOUNDS);
    *a.n_free_out = n_free + F - K;
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
      int begun_page = -1;
      int64_t base = 0;
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        const int t = t0 + u;
        slot[u] = -1;
        if (t >= n_tok) continue;
        if (t >= end) {
          b = find_last(s_tok, a.B, t);
          end = b + 1 < a.B ? s_tok[b + 1] : n_tok;
          begun_page = stop ? -1 : s_begun[b];
          cur = s_cur[b];
          tb = s_tok[b];
          page_b = s_need[b] - pages(cur);
          col = -1;
        }
        if (begun_page < 0) continue;
        const int pos = cur + (t - tb);
        if (pos >> sh != col) {
          col = pos >> sh;
          const int page = col < pages(cur) ? begun_page : taken_page(page_b + col);
          base = (int64_t)page << sh;
        }
        slot[u] = base + (pos & (int)page_mask);
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
      a.table[(size_t)b * a.W + pages(s_cur[b]) + (k - s_need[b])] = taken_page(k);
      continue;
    }
    y -= K;
    if (y < kept) {
      // position n_free + y of the stack
      a.free_pages[n_free + (int)y] = taken_page(F - 1 - (int)y);
      continue;
    }
    const int b = (int)(y - kept);
    a.out_lens[b] = !stop && s_begun[b] >= 0 ? s_new[b] : s_cur[b];
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
  const int smem = (6 * a.B + std::min(a.n_pages, kResizeIds)) * (int)sizeof(int);
  constexpr int kMost = (6 * kResizeSeqs + kResizeIds) * (int)sizeof(int);
  static_assert(kMost <= 227 * 1024 - 2048, "batch exceeds shared memory");
  static DeviceOnce once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMost);
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
