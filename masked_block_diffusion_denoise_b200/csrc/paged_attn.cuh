// Parts shared by the paged attention kernels (bf16 on the tensor cores, float32
// on the CUDA cores): what a row sees, how the work is cut into one range per
// CTA, the walk over a range's items, and the join of items that were cut.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "kernels.h"

namespace dlm {

namespace {

constexpr int kSlotRows = 256;   // rows of a partial in the workspace

// two float32 in one register pair (sm_100 packed arithmetic)
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A piece of work: up to `positions` consecutive positions of a sequence for one
// KV head (with that head's G query heads), and a range of their key tiles.
struct Item {
  int b, g;
  int row0, npos;      // first row of q, positions of the item
  int pos0, ctx;       // position of the first row, keys of the sequence
  int ts, te;          // key tiles of this CTA
  int kt0, pair;       // key tiles of row tile 0; two row tiles
  int whole;           // every key tile is here: write the result
  int slot;            // partial slot (1: the item starts here)
  int fix;             // keys that every row sees; V behind them is checked
  int poison;          // ... and holds an infinity or NaN
  int valid;           // 0: no more items
  int pad;
};
static_assert(sizeof(Item) == 64, "");

// What the join needs to know of a CTA's cut items
struct Meta {
  int tail;            // an item starts here and is cut
  int row0, npos, g, pair;
  int head;            // a partial of an item that started earlier
  int head_ends;       // ... whose last key tile is here
  int pos0;            // position of row0
};

struct Params {
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* table;
  const void* k;
  const void* v;
  const void* q;
  int64_t q_stride;
  void* o;
  int64_t o_stride;
  float* lse;
  float* part;         // [cta][2][kSlotRows x Dh], order: part_at
  float2* ml;          // [cta][2][kSlotRows]
  Meta* meta;          // [cta]
  int* err;
  int W, B, T, H, Hkv, G, npos, block, n_pages, page_shift;
  int positions;       // of an item: npos, or 2 * npos (two row tiles)
  uint32_t g_inv;      // ceil(2^16 / G): x / G for x < 256
  double inv_grid;     // 1 / CTAs
  float scale_log2;
};

__device__ __noinline__ int block_end(int p, int ctx, int block) {
  return (int)min((long long)ctx, ((long long)(p / block) + 1) * block);
}
// what a row's sum of products is multiplied by: zeros for a row that sees no key,
// 0 x infinity for one that does and has only scores of -infinity
__device__ __forceinline__ float inverse(float l, bool sees) { return sees ? 1.f / l : 0.f; }
// keys [0, n) that the row at position p sees
__device__ __forceinline__ int visible(int p, int ctx, int block) {
  if (block == 0) return ctx;
  if (p < 0) return 0;
  if (block == 1) return min(ctx, p + 1);
  return block_end(p, ctx, block);
}

// The cost of a sequence's items, in keys: item j (pp positions) costs the keys
// below its last row's position (its block's end is not counted) plus item_cost
// (loading Q, the first scores, the results).  cum(j) is the cost of the items before j.
struct SeqCost {
  long long base;   // position of row 0
  int n, ctx, pp, items, j0;
  long long item_cost;
  bool masked;
  __device__ SeqCost(int n_, int ctx_, int pp_, int block, int cost)
      : base((long long)ctx_ - n_), n(n_), ctx(ctx_), pp(pp_), item_cost(cost), masked(block != 0) {
    items = (int)(((uint32_t)n + (uint32_t)pp - 1u) / (uint32_t)pp);
    // items wholly before position 0 (masked, base < 0): no keys
    j0 = base < 0 ? min(max(items - 1, 0), (int)(-base / pp)) : 0;
  }
  __device__ long long cum(int j) const {
    if (!masked) return (long long)j * (ctx + item_cost);
    const bool end = j == items && j > 0;
    if (end) --j;
    long long c = item_cost * j;
    if (j > j0)
      c += (j - j0) * base +
           (long long)pp * (((long long)j * (j + 1) - (long long)j0 * (j0 + 1)) / 2);
    if (end) c += ctx + item_cost;
    return c;
  }
};

// x / G for 0 <= x < 256, G <= 128: the rounded-up factor adds less than
// 2^8 / 2^16 to the quotient, and its fraction is at most 1 - 2^-7
__device__ __forceinline__ int div_g(const Params& p, int x) {
  return (int)(((uint32_t)x * p.g_inv) >> 16);
}

// Offsets ascending within the rows, a length that the table can hold (and that
// leaves room for a tile's end in 32 bits).  cu, ctx and table are read with
// plain loads: the kernel before, which may write them, can still run when this
// one starts, so they are not read-only for its whole life.
__device__ __forceinline__ bool seq_ok(const Params& p, int c0, int c1, int ctx) {
  return c0 >= 0 && c0 <= c1 && c1 <= p.T && ctx >= 0 && ctx <= 0x7FFF0000 &&
         (long long)ctx <= ((long long)p.W << p.page_shift);
}

// The block's exclusive scans of x and y; the sums in *all.  `scan`: shared
// memory, a pair per warp.
template <int THREADS>
__device__ __forceinline__ longlong2 block_scan(longlong2 x, longlong2* scan, longlong2* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  longlong2 incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, incl.x, d);
    const long long b = __shfl_up_sync(0xffffffffu, incl.y, d);
    if (lane >= d) {
      incl.x += a;
      incl.y += b;
    }
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  longlong2 before = make_longlong2(0, 0);
  *all = make_longlong2(0, 0);
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = *all;
    all->x += scan[w].x;
    all->y += scan[w].y;
  }
  return make_longlong2(before.x + incl.x - x.x, before.y + incl.y - x.y);
}

// the page ids of a sequence from key k on are needed soon
__device__ __forceinline__ void prefetch_pages(const Params& p, int b, int k) {
  const int col = min(k >> p.page_shift, p.W - 1);
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p.table + (size_t)b * p.W + col));
}

// u / w, by a double's quotient and a correction (u < 2^53)
__device__ __forceinline__ int small_quotient(long long u, long long w) {
  int g = (int)((double)u * __drcp_rn((double)w));
  g -= g * w > u;
  g += (g + 1) * w <= u;
  return g;
}

// This CTA's range of the work, as (KV head, sequence, item, key tile) in start
// and stop ([0] = Hkv: the end).  A scan over the sequences, consecutive ones per
// thread; the owners of the range's two ends turn them into an item and a tile.
//   Little work (every item cut into pieces of min_tiles key tiles gives no more
//   pieces than CTAs): a piece per CTA, so that none has two items.
//   Else all items, KV head by KV head, are laid end to end in units of cost
//   and cut into equal shares.
// `scan`: shared memory, a pair of numbers per warp.  The caller synchronises before
// it reads start and stop.
template <int THREADS>
__device__ void find_range(const Params& p, int key_tile, int item_cost, int min_tiles,
                           longlong2* scan, int* start, int* stop) {
  const int tid = threadIdx.x;
  const int pp = p.positions;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  // the sequence's new tokens and length; none if the input is bad
  auto sequence = [&](int b, int& n, int& ctx, bool report) {
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    ctx = p.ctx[b];
    n = c1 - c0;
    if (!seq_ok(p, c0, c1, ctx)) {
      if (report) raise_error(p.err, DLM_EBOUNDS);
      n = ctx = 0;
    }
  };
  // key tiles of item j of a sequence
  auto tiles = [&](int n, int ctx, int j) {
    const int i1 = min(n, (j + 1) * pp);
    return (visible(ctx - n + i1 - 1, ctx, p.block) + key_tile - 1) / key_tile;
  };
  // pieces of min_tiles key tiles
  auto pieces = [&](int n, int ctx, int j) {
    return max(1, (tiles(n, ctx, j) + min_tiles - 1) / min_tiles);
  };
  if (tid < 4) start[tid] = stop[tid] = 0;
  // a sequence's cost, and its pieces unless its keys or items alone make more than the grid
  const long long few = (long long)gridDim.x * min_tiles * key_tile;
  longlong2 own = make_longlong2(0, 0), sum;
  for (int b = b0; b < b1; ++b) {
    int n, ctx;
    sequence(b, n, ctx, blockIdx.x == 0);
    const SeqCost s(n, ctx, pp, p.block, item_cost);
    const long long c = s.cum(s.items);
    own.x += c;
    if ((c - (long long)s.items * item_cost) * p.Hkv > few || own.y > gridDim.x ||
        s.items > (int)gridDim.x)
      own.y = gridDim.x + 1;
    else
      for (int j = 0; j * pp < n; ++j) own.y += pieces(n, ctx, j);
  }
  const longlong2 before = block_scan<THREADS>(own, scan, &sum);
  const long long mine = own.x, first = before.x, w1 = sum.x, total = w1 * p.Hkv;
  {
    const long long all = sum.y;
    if (all * p.Hkv <= gridDim.x) {
      if ((int)blockIdx.x >= all * p.Hkv) {
        if (tid == 0) start[0] = stop[0] = p.Hkv;
        return;
      }
      const int g = (int)blockIdx.x / (int)all;
      int r = (int)blockIdx.x - g * (int)all - (int)before.y;
      if (r < 0 || r >= own.y) return;
      for (int b = b0; b < b1; ++b) {
        int n, ctx;
        sequence(b, n, ctx, false);
        for (int j = 0; j * pp < n; ++j) {
          const int k = pieces(n, ctx, j);
          if (r < k) {
            prefetch_pages(p, b, r * min_tiles * key_tile);
            start[0] = stop[0] = g;
            start[1] = stop[1] = b;
            start[2] = j;
            start[3] = r * min_tiles;
            stop[2] = r + 1 < k ? j : j + 1;
            stop[3] = r + 1 < k ? (r + 1) * min_tiles : 0;
            return;
          }
          r -= k;
        }
      }
      return;
    }
  }
  // (a share rounded up: the last CTAs may have none)
  const long long share = (long long)((double)total * p.inv_grid) + 1;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int* dst = e == 0 ? start : stop;
    const long long u = min(total, share * ((int)blockIdx.x + e));
    if (u >= total) {
      if (tid == 0) dst[0] = p.Hkv;   // the end
      continue;
    }
    const int g = small_quotient(u, w1);
    long long r = u - g * w1 - first;
    if (r < 0 || r >= mine) continue;
    for (int b = b0; b < b1; ++b) {
      int n, ctx;
      sequence(b, n, ctx, false);
      const SeqCost s(n, ctx, pp, p.block, item_cost);
      const long long c = s.cum(s.items);
      if (r >= c) {
        r -= c;
        continue;
      }
      int lo = 0, hi = s.items;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.cum(mid) <= r)
          lo = mid;
        else
          hi = mid;
      }
      // the share of the item's cost, as key tiles: < kt; 0: the item starts in
      // the range behind this edge
      const float at = (float)(r - s.cum(lo)), cost = (float)(s.cum(lo + 1) - s.cum(lo));
      const int kt = tiles(n, ctx, lo);
      if (e == 0) prefetch_pages(p, b, (int)__fdividef(at * kt, cost) * key_tile);
      dst[0] = g;
      dst[1] = b;
      dst[2] = lo;
      dst[3] = max(0, min(kt - 1, (int)__fdividef(at * kt, cost)));
      break;
    }
  }
}

// The items of a range in order; every lane of a warp gets the same item.  meta
// collects what the join needs of the items that the range cuts.
struct Walker {
  int g, b, j, t0, g1, b1, j1, t1;
  int cb = -1, l0 = 0, l1 = 0, lc = 0;   // 32 sequences, one per lane
  Meta meta = {};
  __device__ Walker(const int* start, const int* stop)
      : g(start[0]), b(start[1]), j(start[2]), t0(start[3]), g1(stop[0]), b1(stop[1]), j1(stop[2]),
        t1(stop[3]) {}
  __device__ Item next(const Params& p, int key_tile, int lane) {
    for (;;) {
      Item it = {};
      if (!(g < g1 || (g == g1 && g < p.Hkv &&
                       (b < b1 || (b == b1 && (j < j1 || (j == j1 && t1 > 0)))))))
        return it;
      if (b >> 5 != cb) {
        cb = b >> 5;
        const int bb = cb * 32 + lane;
        const bool in = bb < p.B;
        l0 = in ? p.cu[bb] : 0;
        l1 = in ? p.cu[bb + 1] : 0;
        lc = in ? p.ctx[bb] : 0;
        if (!in || !seq_ok(p, l0, l1, lc)) l1 = l0 = 0;
      }
      const int c0 = __shfl_sync(0xffffffffu, l0, b & 31);
      const int c1 = __shfl_sync(0xffffffffu, l1, b & 31);
      const int ctx = __shfl_sync(0xffffffffu, lc, b & 31);
      const int len = c1 - c0;
      if ((long long)j * p.positions >= len) {   // the next sequence, then the next KV head
        j = 0;
        t0 = 0;
        // over the empty sequences of these 32 at once
        const uint32_t full = __ballot_sync(0xffffffffu, l1 > l0);
        const uint32_t later = (b & 31) == 31 ? 0u : full & (0xffffffffu << ((b & 31) + 1));
        b = later != 0 ? (b & ~31) + __ffs(later) - 1 : (b & ~31) + 32;
        if (b >= p.B) {
          b = 0;
          ++g;
        }
        continue;
      }
      const int i0 = j * p.positions;
      it.b = b;
      it.g = g;
      it.row0 = c0 + i0;
      it.npos = min(p.positions, len - i0);
      it.pos0 = ctx - len + i0;
      it.ctx = ctx;
      it.pair = it.npos > p.npos;
      const int last0 = it.pos0 + min(it.npos, p.npos) - 1;
      it.kt0 = (visible(last0, ctx, p.block) + key_tile - 1) / key_tile;
      const int kt = (visible(it.pos0 + it.npos - 1, ctx, p.block) + key_tile - 1) / key_tile;
      const bool stops = g == g1 && b == b1 && j == j1;
      it.ts = t0;
      it.te = stops ? t1 : kt;
      it.whole = it.ts == 0 && it.te == kt;
      it.slot = it.ts == 0;
      it.fix = visible(it.pos0, ctx, p.block);
      it.valid = 1;
      const bool nothing = !it.whole && it.ts >= it.te;   // no tile of a cut item
      if (!it.whole) {
        if (it.ts == 0) {
          meta.tail = 1;
          meta.row0 = it.row0;
          meta.pos0 = it.pos0;
          meta.npos = it.npos;
          meta.g = g;
          meta.pair = it.pair;
        } else {
          meta.head = !nothing;
          meta.head_ends = it.te == kt;
        }
      }
      t0 = 0;
      ++j;
      if (!nothing) return it;
    }
  }
};

// Where column `col` of row `row` of a partial lies, in floats.  The bf16 kernel's
// writers hold a row per lane: four columns of all rows, then the next four, so
// that their 16-byte stores fill whole lines (row after row they touched 32 lines
// each: canvas of 32 tokens, 32 heads 17.7 us instead of 16.6 for the call).  The
// float32 kernel's threads hold a row's columns side by side: row after row (22.8 us
// for its chunks of up to 96 tokens, 23.7 the other way).
template <typename T, int DH>
__device__ __forceinline__ size_t part_at(size_t slot, int row, int col) {
  if (std::is_same<T, float>::value) return (slot * kSlotRows + row) * DH + col;
  return ((slot * (DH / 4) + (col >> 2)) * kSlotRows + row) * 4 + (col & 3);
}

// Joins the partials of an item that starts in CTA c: c's own, then those of
// c + 1, ... up to the CTA where it ends, in that order.  A warp takes 8 rows x 16
// columns, four columns a lane, and kBatch partials at a time: their maxima,
// sums and columns are all loaded before any is used, since the join is a chain
// of loads and it is the number of links that counts.
template <typename T, int DH>
__global__ void __launch_bounds__(256) paged_join_kernel(const Params p, int n_ctas) {
  constexpr int kRowWarps = DH / 16, kGroups = 8 / kRowWarps, kBatch = 8;
  constexpr int kTileRows = kSlotRows / 2;
  pdl_wait_then_release();
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Meta me = p.meta[c];
  // the CTAs behind c, 32 at a time in the lanes: those with a partial of the item,
  // and up to which one it goes
  uint32_t heads, upto;
  bool ends;
  auto look = [&](int k0) {
    const int k = k0 + lane;
    const bool in = k < n_ctas && k > c;
    const int head = in ? p.meta[k].head : 0, last = in ? p.meta[k].head_ends : 0;
    const uint32_t stops = __ballot_sync(0xffffffffu, last != 0);
    ends = stops != 0 || k0 + 32 >= n_ctas;
    upto = stops != 0 ? 0xffffffffu >> (32 - __ffs(stops)) : 0xffffffffu;
    heads = (__ballot_sync(0xffffffffu, head != 0) | (k0 == c ? 1u : 0u)) & upto;
  };
  // rows in use of row tile `tile`: its first ones
  auto used = [&](int tile) { return min(p.npos, me.npos - tile * p.npos) * p.G; };
  // blocks without rows leave before they look further (the first one has some,
  // and looks while it waits for `me`)
  const int first = blockIdx.y * kGroups * 8;
  if (first > 0 && (!me.tail || (!me.pair && first >= used(0)))) return;
  look(c);
  if (!me.tail) return;
  const int col = (warp % kRowWarps) * 16 + (lane >> 3) * 4;
  for (int g = blockIdx.y * kGroups + warp / kRowWarps; g < kSlotRows / 8;
       g += gridDim.y * kGroups) {
    const int row = g * 8 + (lane & 7), tile = row / kTileRows, x = row - tile * kTileRows;
    const bool live = x < used(tile);
    if (!__any_sync(0xffffffffu, live)) continue;
    float m = -CUDART_INF_F, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = c;; k0 += 32) {
      if (k0 > c || g >= (int)gridDim.y * kGroups) look(k0);   // (done for the first group)
      for (uint32_t rest = heads; rest != 0;) {
        float2 v[kBatch];
        float4 y[kBatch];
        float bm = m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          v[u] = make_float2(-CUDART_INF_F, 0.f);
          y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (rest == 0 || !live) continue;
          const int k = k0 + __ffs(rest) - 1;
          rest &= rest - 1;
          const size_t slot = (size_t)k * 2 + (k == c);
          v[u] = p.ml[slot * kSlotRows + row];
          y[u] = *reinterpret_cast<const float4*>(p.part + part_at<T, DH>(slot, row, col));
        }
        if (!live) rest = 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) bm = fmaxf(bm, v[u].x);
        const float base = bm == -CUDART_INF_F ? 0.f : bm;   // no key seen so far
        const float old = fast_exp2(m - base);
        l *= old;
        acc.x *= old;
        acc.y *= old;
        acc.z *= old;
        acc.w *= old;
        m = bm;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          // A part without a key of this row has l and columns of 0.  None is passed
          // over for a weight of 0: where every score was NaN the maximum is -inf and
          // l is NaN, and that has to reach the result, as it does in an item that is not cut.
          const float w = fast_exp2(v[u].x - base);
          l = fmaf(w, v[u].y, l);
          acc.x = fmaf(w, y[u].x, acc.x);
          acc.y = fmaf(w, y[u].y, acc.y);
          acc.z = fmaf(w, y[u].z, acc.z);
          acc.w = fmaf(w, y[u].w, acc.w);
        }
      }
      if (ends) break;
    }
    if (!live) continue;
    const int rp = div_g(p, x), rh = x - rp * p.G, pos = tile * p.npos + rp;
    // (an item that is cut has keys: only a mask can hide them all)
    const float inv = inverse(l, p.block == 0 || me.pos0 + pos >= 0);
    const int64_t grow = (int64_t)me.row0 + pos;
    const int head = me.g * p.G + rh;
    T* dst = (T*)p.o + grow * p.o_stride + (int64_t)head * DH + col;
    if constexpr (std::is_same<T, float>::value) {
      *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
      __nv_bfloat162 r[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                             __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(r);
    }
    if (p.lse != nullptr && col == 0)
      p.lse[(size_t)grow * p.H + head] =
          l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
  }
}

inline size_t part_bytes(int ctas, int Dh) {
  return (size_t)ctas * 2 * kSlotRows * Dh * sizeof(float);
}
inline size_t ml_bytes(int ctas) { return (size_t)ctas * 2 * kSlotRows * sizeof(float2); }
inline size_t work_bytes(int ctas, int Dh) {
  return part_bytes(ctas, Dh) + ml_bytes(ctas) + (size_t)ctas * sizeof(Meta);
}

inline Params make_params(const PagedAttn& a, int ctas) {
  Params p;
  p.cu = a.cu;
  p.ctx = a.ctx;
  p.table = a.table;
  p.k = a.c.k;
  p.v = a.c.v;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.o = a.o;
  p.o_stride = a.o_stride;
  p.lse = a.lse;
  uint8_t* work = (uint8_t*)a.work;
  p.part = (float*)work;
  p.ml = (float2*)(work + part_bytes(ctas, a.c.Dh));
  p.meta = (Meta*)(work + part_bytes(ctas, a.c.Dh) + ml_bytes(ctas));
  p.err = a.err;
  p.W = a.W;
  p.B = a.B;
  p.T = a.T;
  p.H = a.H;
  p.Hkv = a.c.Hkv;
  p.G = a.H / a.c.Hkv;
  p.block = a.block;
  p.n_pages = a.c.n_pages;
  p.page_shift = a.c.page_shift;
  p.g_inv = (65536u + (uint32_t)p.G - 1u) / (uint32_t)p.G;
  p.inv_grid = 1.0 / ctas;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  return p;
}

// `rows`: of a slot at most.  Blocks per CTA's item for half as many rows again as a
// sequence's tokens make on average, so that few are launched for nothing; longer
// items loop.  (us a call: single tokens of 61 sequences, 4 rows an item, blocks for 256
// rows 121.2, for 8 119.4; canvases of 32 over 32768 keys, 128 rows, for 256 105.0, for 128
// 103.3; one canvas of 32 over 2048, for all 128 16.5, for 64 and less 21.0; float32 chunks
// of 1..96 tokens, for 64 rows 22.5, for their mean 23.8; causal chunks of up to 4096: no
// difference.)
template <typename T, int DH>
cudaError_t launch_join(const Params& p, int ctas, int rows, cudaStream_t st) {
  constexpr int kBlockRows = 8 * (8 / (DH / 16));
  const long long tokens = min((long long)p.T, (3ll * p.T + 2 * p.B - 1) / (2 * p.B));
  rows = (int)min((long long)rows, tokens * p.G);
  const int blocks = (rows + kBlockRows - 1) / kBlockRows;
  return launch_pdl(paged_join_kernel<T, DH>, dim3(ctas, blocks), dim3(256), 0, st, p,
                    ctas);
}

}  // namespace

}  // namespace dlm
