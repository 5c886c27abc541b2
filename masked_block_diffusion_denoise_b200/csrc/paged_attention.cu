// bf16 attention of ragged chunks of new tokens over a paged KV cache.
//
// Rows.  The G = H / Hkv query heads of a KV head share its keys: a row tile is
// npos = floor(128 / G) positions x G heads (row = position * G + head), at
// most 128 rows = the M of the tensor core's tiles; an item is two
// consecutive row tiles of a sequence for one KV head.  An item whose second
// row tile is empty (single tokens, short chunks) gives every other key tile
// to the second half of the CTA instead, with the same queries.
//
// Work.  The grid is persistent, one CTA per SM.  All items, laid end to end in
// units of keys, are cut into equal ranges, one per CTA, so that one long
// sequence spreads over all SMs and many short ones share them; lengths are
// read on the device.  An item that lies in one range is written as bf16; one
// that is cut leaves float32 partials (unnormalised O, running maximum and
// sum) in the workspace, which a second kernel joins in a fixed order.
//
// Pages.  K and V pages come by TMA as a 5-D box (64 dims, 8 rows, Dh / 64
// halves, rows / 8 groups, 1 page): whatever the page size (>= 8), a 128-key
// tile in shared memory is [16 groups of 8 rows][half][8 rows][128 bytes], with
// one stride between 8-row groups, which is what the MMA descriptors need.
//
// What bounds it (32 query / 8 KV heads x 128 unless said otherwise; a call from
// Python, and in a graph of ten):
//   single tokens of 61 sequences over 1024..4096 keys: HBM, 655 MB in 138 us, 4.7
//   TB/s (120 us, 5.5); range, first pages and first tile take 7 us of it;
//   canvases of 32 over 32768 keys: HBM, 540 MB in 122 us, 4.4 TB/s (104 us, 5.2);
//   chunks of up to 4096 over up to 8192 keys, causal: the softmax, 1.33 TFLOP in 1526
//   us, 0.87 PFLOP/s (1317 to 1457), where calls follow each other and the power limit
//   lowers the clock (1262 was the best seen; variants are compared with that).  A pair of 128 x 128 tiles takes 3900 cycles, 1025 of them
//   tensor work and 2090 the exponential unit's: a warp by itself needs 1950 for its
//   128 exponentials a lane, with their loads from and stores to tensor memory (the
//   unit alone 1050), and the two warps of a scheduler side by side need no less
//   than in turns;
//   finished blocks of 256, 16 / 4 heads x 64, 700..1800 new tokens of 3 sequences: the
//   same, 31.6 GFLOP in 79 us (78), 11 of them before the first P;
//   a canvas of 32 over 2048 keys: latency, 16.8 us (16.7): range 2.6, its item and page ids
//   1.6, first tile 0.9, first P 1.9, results 1.3; the rest is the stores of its partials
//   and the join.
//
// Precision: scores, softmax statistics and O are float32; each probability is rounded
// to bf16, the tensor core's operand type, before P V and summed unrounded.  Outputs are
// 0.0020 to 0.0023 off the 64-bit result (2-norm, relative), 0.0017 of it the rounding
// of the result itself.
#include "paged_attn.cuh"

namespace dlm {

DLM_TRACE_STORAGE(paged)

namespace {

constexpr int kKeys = 128;       // keys per tile
constexpr int kRows = 128;       // rows per row tile
// 16 warps: softmax of row tile 0 and 1 (four each), producer, MMA issuers of
// row tile 0 and 1, scheduler, and four that write results (and check V), so
// that the softmax goes on with the next item meanwhile
constexpr int kThreads = 512;
constexpr int kProducer = 8, kMma = 9, kScheduler = 11, kWriter = 12;
constexpr int kDescs = 4;
// Tensor memory: S0, S1 (128 columns each), O0, O1 (Dh each), and P (64 columns of
// bf16 pairs): for Dh 64 in columns of its own, for Dh 128 in the upper half of its
// S, whose lower half is then free for the next S
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
template <int DH>
__device__ __forceinline__ uint32_t col_p(int i) {
  return DH == 64 ? kColO + 128 + i * 64 : i * kKeys + 64;
}
// Cost of an item beside its keys, in keys: loading Q, the first S, the epilogue.
// Finished blocks of 256 tokens (16 / 4 heads x 64), causal chunks of up to 4096 (32 / 8
// x 128), us: 32 keys 77.7 and 1285, 64 76.6 and 1279, 128 74.8 and 1269, 256 76.8 and 1243.
constexpr int kItemCost = 128;
// Key tiles of a piece when there is little work.  A canvas of 32 over 2048 keys
// (32 / 8 heads x 128), with the join: one tile 17.4 us (more to join), two 16.5; four 1.6 us
// more than two.
constexpr int kMinTiles = 2;
// the running reference of a row moves only when its maximum passes it by
// more than this (log2 units): P stays below 2^8, O is rarely rescaled
constexpr float kRescaleLog2 = 8.0f;

template <int DH>
struct Tile {
  static constexpr int kHalves = DH / 64;
  static constexpr int kGroup = kHalves * 1024;          // 8 rows
  static constexpr int kBytes = 16 * kGroup;             // a 128-row K or V tile
  static constexpr int kQHalf = kRows * 128;
  static constexpr int kQBytes = kHalves * kQHalf;
  static constexpr int kSlots = DH == 128 ? 5 : 10;      // ring of K and V tiles
};

template <int DH>
struct Smem {
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * Tile<DH>::kQBytes;
  static constexpr int kTail = kRing + Tile<DH>::kSlots * Tile<DH>::kBytes;
  struct Rest {
    Item item[kDescs];
    float2 stat[2][kRows];   // (max, sum) of the rows, per row tile or half
    uint64_t full[Tile<DH>::kSlots], empty[Tile<DH>::kSlots];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], o_empty[2], turn[2][4], pv_done[2];
    uint64_t d_full[kDescs], d_empty[kDescs];
    uint64_t stat_full[2], stat_empty[2], fix_req[2], fix_done[2], fin[2];
    int start[4], stop[4];
    uint32_t tmem;
    int abort;
  };
  static constexpr int kBytes = kTail + (int)sizeof(Rest);
};
static_assert(Smem<128>::kBytes <= 232448 && Smem<64>::kBytes <= 232448, "shared memory");

// matrix descriptors of a 128-row tile whose 8-row groups are `group` bytes
// apart (128-byte swizzle): K-major (rows = N), and MN-major (rows = K, 64-element
// chunks of N 1024 bytes apart)
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr, int group) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(group >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, int group) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(1024 >> 4) << 16 |
         (uint64_t)(group >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int group, int plane) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(plane), "r"(smem_u32(bar))
      : "memory");
}

// Waits of the inner loops: little code (the roles share the instruction
// caches), bounded by the number of tries, each at most about 2 us long.
constexpr uint32_t kTries = 1u << 20;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  for (uint32_t n = 0; !mbar_try_wait_hint(bar, parity, 2000u); ++n) {
    if (n >= kTries) *abort_flag = 1;
    if (*abort_flag) return false;
  }
  return true;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

__device__ __forceinline__ float fmax3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Adds to o (16 columns from c0) the non-finite V elements of keys [k0, k1): the
// V check set them to zero in shared memory, so that rows that do not see
// those keys stay clean.
template <int DH>
__device__ __noinline__ void add_poison(const Params& p, const Item& it, int k0, int k1, int c0,
                                        float* o) {
  const int mask = (1 << p.page_shift) - 1;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    const int page = p.table[(size_t)it.b * p.W + (k >> p.page_shift)];
    if (page < 0 || page >= p.n_pages) continue;
    const __nv_bfloat16* row =
        (const __nv_bfloat16*)p.v + ((((size_t)page * p.Hkv + it.g) << p.page_shift) + (k & mask)) * DH + c0;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
      const float x = __bfloat162float(row[j]);
      if (!(fabsf(x) <= 3.4e38f)) o[j] += x;
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ, const Params p) {
  using TL = Tile<DH>;
  constexpr int NS = TL::kSlots;
  // timeline marks: 2 range known, 3 first K tile, 4 first S, 5 first P written,
  // 6 first O complete, 7 last item done
  DLM_TRACE_CTA(TRACE_PAGED);
  // the tiles' swizzle wants 1024-byte alignment, and there is no room to round up
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {
    pdl_wait_then_release();
    if (threadIdx.x == 0) {
      raise_error(p.err, DLM_EBOUNDS);
      p.meta[blockIdx.x] = Meta{};   // nothing to join
    }
    return;
  }
  uint8_t* qs = smem + Smem<DH>::kQ;
  uint8_t* ring = smem + Smem<DH>::kRing;
  auto& sh = *reinterpret_cast<typename Smem<DH>::Rest*>(smem + Smem<DH>::kTail);
  volatile int* abort_flag = &sh.abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 2);   // both MMA issuers
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 2);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i][0], 4);   // the first 64 keys' P, the others'
      mbar_init(&sh.p_full[i][1], 4);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.o_empty[i], 4);
      mbar_init(&sh.stat_full[i], 4);
      mbar_init(&sh.stat_empty[i], 4);
      mbar_init(&sh.fix_req[i], 2);
      mbar_init(&sh.fin[i], 1);
      mbar_init(&sh.fix_done[i], 4);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&sh.turn[i >> 2][i & 3], 1);
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], 15);   // all warps but the scheduler
    }
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch(&tmK);
    tma_prefetch(&tmV);
    tma_prefetch(&tmQ);
  }
  if (warp == kMma) tmem_alloc(&sh.tmem, kTmemCols);
  // the kernel before this one is waited for here; the join may be set up while
  // this grid runs (it waits for the grid's end)
  pdl_wait_then_release();

  // ---- this CTA's range of the work (the scan's scratch is the ring, free until
  // the first load) ----
  find_range<kThreads>(p, kKeys, kItemCost, kMinTiles, reinterpret_cast<longlong2*>(ring), sh.start,
                       sh.stop);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (tid == 0) DLM_TRACE_MARK(2);

  if (warp >= kProducer) {
    if (warp == kProducer) {
      // ---------------- producer: Q, K and V tiles ----------------
      uint32_t e = 0;        // ring entries issued (K, V, K, V, ...)
      uint32_t qn = 0;       // Q tiles issued
      bool ok = true;
      const int pages_tile = p.page_shift >= 7 ? 1 : kKeys >> p.page_shift;
      const int page_bytes = TL::kBytes / pages_tile;
      for (uint32_t n = 0; ok; ++n) {
        const int ds = n % kDescs;
        if (!mbar_wait_bounded(&sh.d_full[ds], (n / kDescs) & 1, abort_flag)) break;
        const Item& it = sh.item[ds];
        if (!it.valid) break;
        const int b = it.b, g = it.g, ts = it.ts, te = it.te, ctx = it.ctx;
        const int row0 = it.row0, q_tiles = ts == te ? 0 : it.pair ? 2 : 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.d_empty[ds]);
        const int32_t* row = p.table + (size_t)b * p.W;
        const int n_pages = (ctx + (1 << p.page_shift) - 1) >> p.page_shift;
        int chunk = -1, id = 0, id_next = 0;
        auto load_ids = [&](int c) {
          const int i = c * 32 + lane;
          return i < n_pages ? row[i] : 0;
        };
        for (int t = ts; t < te && ok; ++t) {
          // page ids, 32 at a time, the next 32 on their way
          const int page0 = (int)(((long long)t * kKeys) >> p.page_shift);
          if (page0 >> 5 != chunk) {
            const int c = page0 >> 5;
            id = c == chunk + 1 && chunk >= 0 ? id_next : load_ids(c);
            id_next = load_ids(c + 1);
            chunk = c;
          }
          int page = __shfl_sync(0xffffffffu, id, (page0 + lane) & 31);
          const bool mine = lane < pages_tile && page0 + lane < n_pages;
          if (mine && (page < 0 || page >= p.n_pages)) {
            raise_error(p.err, DLM_EBOUNDS);
            page = p.n_pages;   // outside the map: zeros
          }
          const int plane = page * p.Hkv + g;
          const int group = p.page_shift > 7 ? (t & ((1 << (p.page_shift - 7)) - 1)) * 16 : 0;
          const uint32_t bytes = (uint32_t)(min(pages_tile, n_pages - page0) * page_bytes);
          if (t == ts) {
            // the item's queries first
            for (int i = 0; i < q_tiles && ok; ++i, ++qn) {
              const int qslot = qn & 1;
              ok = wait(&sh.q_empty[qslot], ((qn >> 1) & 1) ^ 1, abort_flag);
              if (ok && lane == 0) {
                mbar_arrive_expect_tx(&sh.q_full[qslot], (uint32_t)(p.npos * p.G * DH * 2));
                for (int h = 0; h < TL::kHalves; ++h)
                  tma_load_3d(qs + qslot * TL::kQBytes + h * TL::kQHalf, &tmQ, &sh.q_full[qslot],
                              h * 64, g * p.G, row0 + i * p.npos);
              }
            }
            if (!ok) break;
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = e % NS;
            if (!wait(&sh.empty[slot], ((e / NS) & 1) ^ 1, abort_flag)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], bytes);
            __syncwarp();
            if (mine)
              tma_load_5d(ring + slot * TL::kBytes + lane * page_bytes, kv == 0 ? &tmK : &tmV,
                          &sh.full[slot], group, plane);
            ++e;
          }
        }
      }
      if (*abort_flag) {
        // the copies in flight land before the CTA exits
        for (uint32_t k = e > NS ? e - NS : 0; k < e; ++k)
          mbar_wait_bounded(&sh.full[k % NS], (k / NS) & 1, nullptr);
        for (uint32_t k = qn > 2 ? qn - 2 : 0; k < qn; ++k)
          mbar_wait_bounded(&sh.q_full[k & 1], (k >> 1) & 1, nullptr);
      }
    } else if (warp < kScheduler) {
      // ---------------- MMA issuers: one warp per row tile (or half) ----------------
      // In order, per key tile: S_i(l), then P_i(l) V(l).  A wait that follows MMAs
      // in a warp returns only when those have left its queue, and the tensor core
      // would run dry meanwhile (measured: 1375 instead of 1025 cycles for 8 + 8
      // MMAs); with a warp per row tile the other's MMAs fill the gap.  Both warps
      // wait for, and release, every ring entry: a barrier's phases are then seen
      // in order whoever uses the entry.  The whole warp walks the loop and one
      // elected lane issues: operands that are the same in all lanes reach the MMA
      // without a move per instruction.
      const int i = warp - kMma;
      constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
      constexpr uint32_t idesc_h = idesc_bf16_f32(kRows, kKeys / 2);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, DH, true);
      const uint32_t tm_s = __shfl_sync(0xffffffffu, tmem + i * kKeys, 0);
      const uint32_t tm_o = __shfl_sync(0xffffffffu, tmem + kColO + i * DH, 0);
      const uint32_t tm_p = __shfl_sync(0xffffffffu, tmem + col_p<DH>(i), 0);
      const uint64_t kd0 = desc_k(smem_u32(ring), TL::kGroup);
      const uint64_t vd0 = desc_mn(smem_u32(ring), TL::kGroup);
      const uint64_t qd0 = desc_k(smem_u32(qs), 1024);
      uint32_t slot = 0, phase = 0;  // ring
      auto advance = [&]() {
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      };
      uint32_t qn = 0;               // Q tiles used
      uint32_t np = 0, no = 1;       // phases of the next P, of the next wait for an empty O
      uint32_t fb = 0;               // V checks of earlier items
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        const int ds = n % kDescs;
        if (!mbar_wait_bounded(&sh.d_full[ds], (n / kDescs) & 1, abort_flag)) break;
        const Item& it = sh.item[ds];
        if (!__shfl_sync(0xffffffffu, it.valid, 0)) break;
        const int L = __shfl_sync(0xffffffffu, it.te - it.ts, 0);
        const bool pair = __shfl_sync(0xffffffffu, it.pair, 0) != 0;
        // own tiles: first, first + step, ... below limit
        const int first = pair ? 0 : i, step = pair ? 1 : 2;
        const int limit =
            pair && i == 0 ? max(0, min(L, __shfl_sync(0xffffffffu, it.kt0 - it.ts, 0))) : L;
        const int fix_l = max(0, __shfl_sync(0xffffffffu, it.fix / kKeys - it.ts, 0));
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.d_empty[ds]);
        if (L == 0) continue;
        const uint32_t q0 = qn & 1, qi = pair ? q0 ^ i : q0;
        if (!wait(&sh.q_full[q0], (qn >> 1) & 1, abort_flag) ||
            (pair && !wait(&sh.q_full[q0 ^ 1], ((qn + 1) >> 1) & 1, abort_flag)))
          break;
        const uint64_t qd = qd0 + (uint64_t)(qi * (TL::kQBytes >> 4));
        // A Q tile is free again when both issuers have said so, the one that does not
        // use it as soon as it has seen it come: it would otherwise miss the next one
        if (pair && lane == 0) mbar_arrive(&sh.q_empty[qi ^ 1]);
        int own = first;   // the next own tile
        // no tile here (a row tile without keys, a half without a key tile)
        if (own >= limit && lane == 0) mbar_arrive(&sh.q_empty[qi]);
        // S_i = Q_i K^T: all 128 keys, or the lower (part 0) or upper (part 1) 64
        auto issue_s = [&](uint32_t ks, int part) {
          const bool half = part >= 0;
          const uint64_t kd = kd0 + (uint64_t)((ks * TL::kBytes + (part == 1 ? 8 * TL::kGroup : 0)) >> 4);
          const uint32_t d = tm_s + (part == 1 ? 64 : 0), idesc = half ? idesc_h : idesc_s;
#pragma unroll
          for (int x = 0; x < DH / 16; ++x)
            umma_bf16(d, qd + (uint64_t)(((x >> 2) * TL::kQHalf + (x & 3) * 32) >> 4),
                      kd + (uint64_t)(((x >> 2) * 1024 + (x & 3) * 32) >> 4), idesc, x > 0);
        };
        bool k_there = false;   // S(l) is issued already
        for (int l = 0; l < L; ++l) {
          const bool mine = l == own && l < limit;
          const bool last = l + step >= limit;
          if (!k_there && !wait(&sh.full[slot], phase, abort_flag)) {
            ok = false;
            break;
          }
          if (mine && !k_there) {
            tc_fence_after();
            if (elect_one()) {
              issue_s(slot, -1);
              umma_commit(&sh.s_full[i]);
              umma_commit(&sh.empty[slot]);
              if (last) umma_commit(&sh.q_empty[qi]);
              if (l == 0 && n == 0) DLM_TRACE_MARK(3);
            }
          } else if (!mine && lane == 0) {
            mbar_arrive(&sh.empty[slot]);
          }
          // the V check may look at V(l): both issuers are done with what its slot held
          // (and with the check before it, so at most one request is open)
          if (l >= fix_l && lane == 0) mbar_arrive(&sh.fix_req[(fb + (l - fix_l)) & 1]);
          __syncwarp();
          advance();
          if (!wait(&sh.full[slot], phase, abort_flag)) {
            ok = false;
            break;
          }
          // both issuers wait for the V check, the one that does not use this V as well:
          // else it could ask for a check two further on, which would count as the
          // other's request for this one
          if (l >= fix_l) {
            const uint32_t k = fb + (l - fix_l);
            if (!wait(&sh.fix_done[k & 1], (k >> 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
          }
          if (mine) {
            // O_i (+)= P_i(l) V(l)
            if (l == first) {
              ok = ok && wait(&sh.o_empty[i], no, abort_flag);
              no ^= 1;
            }
            // two row tiles: the next K first, so that no wait parts its S from P V
            k_there = pair && !last;
            const uint32_t ks = slot + 1 == NS ? 0 : slot + 1;
            if (k_there) ok = ok && wait(&sh.full[ks], phase ^ (ks == 0 ? 1u : 0u), abort_flag);
            // P V in two halves, the first during the second's exponentials; with the
            // first, what of the next S has room (Dh 64: all of it; Dh 128: its lower
            // half, the upper one after P has been read)
            const uint64_t vd = vd0 + (uint64_t)(slot * (TL::kBytes >> 4));
#pragma unroll 1
            for (int h = 0; h < 2 && ok; ++h) {
              ok = wait(&sh.p_full[i][h], np, abort_flag);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                if (DH == 64 && h == 0 && k_there) {
                  issue_s(ks, -1);
                  umma_commit(&sh.s_full[i]);
                  umma_commit(&sh.empty[ks]);
                }
#pragma unroll
                for (int x = 0; x < kKeys / 32; ++x)
                  umma_bf16_tmem_a(tm_o, tm_p + h * 32 + x * 8,
                                   vd + (uint64_t)((h * 8 + x * 2) * TL::kGroup >> 4), idesc_o,
                                   l != first || h > 0 || x > 0);
                if (DH == 64 && h == 1) umma_commit(&sh.pv_done[i]);
                if (DH == 128 && k_there) {
                  issue_s(ks, h);
                  if (h == 1) {
                    umma_commit(&sh.s_full[i]);
                    umma_commit(&sh.empty[ks]);
                  }
                }
                if (h == 1) {
                  if (k_there && l + 1 + step >= limit) umma_commit(&sh.q_empty[qi]);
                  umma_commit(&sh.empty[slot]);
                  if (last) umma_commit(&sh.o_full[i]);
                }
              }
              __syncwarp();
            }
            np ^= 1;
            if (!ok) break;
            own += step;
          } else if (lane == 0) {
            mbar_arrive(&sh.empty[slot]);
          }
          __syncwarp();
          advance();
        }
        qn += pair ? 2 : 1;
        fb += max(0, L - fix_l);
      }
      __syncwarp();
      if (elect_one()) umma_commit(&sh.fin[i]);   // every MMA issued has finished
      mbar_wait_bounded(&sh.fin[i], 0, nullptr);
    } else if (warp == kScheduler) {
      // ---------------- scheduler: the range's items, one descriptor each ----------------
      Walker walk(sh.start, sh.stop);
      uint32_t n = 0;
      for (;;) {
        const Item it = walk.next(p, kKeys, lane);
        const int ds = n % kDescs;
        if (!mbar_wait_bounded(&sh.d_empty[ds], ((n / kDescs) & 1) ^ 1, abort_flag)) break;
        if (lane == 0) {
          sh.item[ds] = it;
          mbar_arrive(&sh.d_full[ds]);
        }
        ++n;
        if (!it.valid) break;
      }
      if (lane == 0) p.meta[blockIdx.x] = walk.meta;
    } else {
      // ---------------- writers: V check, results ----------------
      // A hidden key has probability 0, but 0 x infinity is NaN: in tiles with hidden
      // keys, rows of V behind the sequence become zero, and so do non-finite
      // elements of keys that only some rows see (added back below to the rows that
      // do).
      const int quad = warp - kWriter;
      const int row = quad * 32 + lane;
      const uint32_t o_col = tmem + ((uint32_t)(quad * 32) << 16) + kColO;
      const int rp = div_g(p, row), rh = row - rp * p.G;   // position and head of the row
      uint32_t eb = 0, done = 0;
      uint32_t no[2] = {0, 0};                         // O accumulations taken
      for (uint32_t n = 0;; ++n) {
        const int ds = n % kDescs;
        if (!mbar_wait_bounded(&sh.d_full[ds], (n / kDescs) & 1, abort_flag)) break;
        Item& it = sh.item[ds];
        if (!it.valid) break;
        const int ts = it.ts, te = it.te, ctx = it.ctx, fix = it.fix, L = te - ts;
        const bool pair = it.pair != 0;
        bool ok = true;
        for (int t = max(ts, fix / kKeys); t < te; ++t) {
          const uint32_t en = eb + 2 * (t - ts) + 1;
          ok = wait(&sh.fix_req[done & 1], (done >> 1) & 1, abort_flag) &&
               wait(&sh.full[en % NS], (en / NS) & 1, abort_flag);
          if (!ok) break;
          uint8_t* tile = ring + (en % NS) * TL::kBytes;
          const int live = min(kKeys, ctx - t * kKeys);   // rows that hold tokens
          // 16-byte pieces: a warp takes kStep rows at a time, four warps in turn
          constexpr int kPieces = TL::kHalves * 8, kStep = 32 / kPieces;
          const int piece = lane % kPieces, r0 = lane / kPieces + quad * kStep;
          auto at = [&](int r) {
            return reinterpret_cast<uint4*>(tile + (r >> 3) * TL::kGroup + (piece >> 3) * 1024 +
                                            (r & 7) * 128 + (piece & 7) * 16);
          };
#pragma unroll 1
          for (int r = live + r0; r < kKeys; r += 4 * kStep) *at(r) = make_uint4(0, 0, 0, 0);
          // exponent bits all ones: the carry reaches the sign bit
          auto hot = [](uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; };
          uint32_t acc = 0;
          const int first = max(0, fix - t * kKeys) + r0;
#pragma unroll 4
          for (int r = first; r < live; r += 4 * kStep) {
            const uint4 w = *at(r);
            acc |= hot(w.x) | hot(w.y) | hot(w.z) | hot(w.w);
          }
          if (__any_sync(0xffffffffu, (acc & 0x80008000u) != 0)) {
#pragma unroll 1
            for (int r = first; r < live; r += 4 * kStep) {
              uint4 w = *at(r);
              uint32_t* c = &w.x;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t h = hot(c[y]);
                c[y] &= (h & 0x80000000u ? 0u : 0xFFFF0000u) | (h & 0x8000u ? 0u : 0xFFFFu);
              }
              *at(r) = w;
            }
            if (lane == 0) it.poison = 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.fix_done[done & 1]);
          ++done;
        }
        if (!ok) break;
        eb += 2 * L;
        // ---- results: row tile 0, then 1; of one tile, the two halves together ----
        const int c0 = pair ? max(0, min(L, it.kt0 - ts)) : (L + 1) >> 1;
        const int c1 = pair ? L : L >> 1;
        const int tiles = pair ? 2 : 1;
        for (int i = 0; i < tiles; ++i) {
          const int c = i == 0 ? c0 : c1;
          const bool two = !pair && c1 > 0;
          ok = wait(&sh.stat_full[i], n & 1, abort_flag) &&
               (pair || wait(&sh.stat_full[1], n & 1, abort_flag)) &&
               (c == 0 || wait(&sh.o_full[i], no[i] & 1, abort_flag)) &&
               (!two || wait(&sh.o_full[1], no[1] & 1, abort_flag));
          if (!ok) break;
          const int pos = pair ? i * p.npos + rp : rp;
          const bool live = rp < p.npos && pos < it.npos;
          const bool whole = it.whole != 0, poison = it.poison != 0;
          float m = sh.stat[i][row].x, l = sh.stat[i][row].y;
          float w0 = 1.f, w1 = 0.f;
          if (two) {
            const float2 x = sh.stat[1][row];
            const float mm = fmaxf(m, x.x);
            w0 = m == -CUDART_INF_F ? 0.f : fast_exp2(m - mm);
            w1 = x.x == -CUDART_INF_F ? 0.f : fast_exp2(x.x - mm);
            l = l * w0 + x.y * w1;
            m = mm;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.stat_empty[i]);
            if (!pair) mbar_arrive(&sh.stat_empty[1]);
          }
          tc_fence_after();
          if (n == 0 && quad == 0 && lane == 0) DLM_TRACE_MARK(6);
          if (whole) {
            // (without any key c is 0 and O is not used)
            const float inv = inverse(l, p.block == 0 || it.pos0 + pos >= 0);
            w0 *= inv;
            w1 *= inv;
          }
          const size_t slot = (size_t)blockIdx.x * 2 + it.slot;
          const int prow = (pair ? i * kRows : 0) + row;
          const int64_t grow = (int64_t)it.row0 + pos;
          const int head = it.g * p.G + rh;
          if (__any_sync(0xffffffffu, live)) {
            uint4* dst_o = reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + grow * p.o_stride + (int64_t)head * DH);
            // 16 columns at a time: little code, which runs once per item
#pragma unroll 1
            for (int y = 0; y < DH / 16; ++y) {
              float o[16];
              {
                uint32_t r0[16], r1[16];
                tmem_ld16_nowait(o_col + i * DH + y * 16, r0);
                if (two) tmem_ld16_nowait(o_col + DH + y * 16, r1);
                tmem_wait_ld();
                // c == 0: no key was seen, and O holds an earlier item's
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] = c > 0 ? __uint_as_float(r0[z]) * w0 : 0.f;
                if (two)
#pragma unroll
                  for (int z = 0; z < 16; ++z) o[z] = fmaf(__uint_as_float(r1[z]), w1, o[z]);
              }
              if (poison && live) {
                const int lim = visible(it.pos0 + pos, ctx, p.block);
                float x[16];
#pragma unroll
                for (int z = 0; z < 16; ++z) x[z] = o[z];
                add_poison<DH>(p, it, max(ts * kKeys, fix), min(lim, te * kKeys), y * 16, x);
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] = x[z];
              }
              if (live && whole) {
#pragma unroll
                for (int z = 0; z < 2; ++z)
                  dst_o[y * 2 + z] =
                      make_uint4(pack_bf16(o[8 * z], o[8 * z + 1]), pack_bf16(o[8 * z + 2], o[8 * z + 3]),
                                 pack_bf16(o[8 * z + 4], o[8 * z + 5]), pack_bf16(o[8 * z + 6], o[8 * z + 7]));
              } else if (live) {
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  *reinterpret_cast<float4*>(p.part + part_at<__nv_bfloat16, DH>(slot, prow, y * 16 + z * 4)) =
                      make_float4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
              }
            }
            if (live && !whole)
              p.ml[slot * kSlotRows + prow] = make_float2(m, l);
            else if (live && p.lse != nullptr)
              p.lse[(size_t)grow * p.H + head] =
                  l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (c > 0) mbar_arrive(&sh.o_empty[i]);
            if (two) mbar_arrive(&sh.o_empty[1]);
          }
        }
        if (!ok) break;
        no[0] += c0 > 0;
        no[1] += c1 > 0;
        if (lane == 0) mbar_arrive(&sh.d_empty[ds]);
      }
      if (quad == 0 && lane == 0) DLM_TRACE_MARK(7);
    }
  } else {
    // ---------------- softmax: one row per thread ----------------
    const int i = warp >> 2;                          // row tile
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_col = lane_addr + i * kKeys;
    const uint32_t o_col = lane_addr + kColO + i * DH;
    const uint32_t p_col = lane_addr + col_p<DH>(i);
    const int rp = div_g(p, row);                     // position of the row
    uint32_t ns = 0;                                  // S tiles taken
    uint32_t nt = 0;                                  // phase of the next turn
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const int ds = n % kDescs;
      if (!mbar_wait_bounded(&sh.d_full[ds], (n / kDescs) & 1, abort_flag)) break;
      const Item& it = sh.item[ds];
      if (!it.valid) break;
      const bool pair = it.pair != 0;
      const int L = it.te - it.ts;
      const int c0 = pair ? max(0, min(L, it.kt0 - it.ts)) : (L + 1) >> 1;
      const int c1 = pair ? L : L >> 1;
      const int c = i == 0 ? c0 : c1;
      const int pos = pair ? i * p.npos + rp : rp;
      const bool live = rp < p.npos && pos < it.npos;
      const int lim = live ? visible(it.pos0 + pos, it.ctx, p.block) : 0x7fffffff;
      const int lim_min = __reduce_min_sync(0xffffffffu, lim);
      const bool any = __any_sync(0xffffffffu, live);
      // The two row tiles (halves) take turns at the exponentials, each warp with
      // the one that shares its scheduler.  Left alone they fall into step, both
      // at the exponential unit and then both at the tensor core (chunks of up to
      // 4096 tokens, 32 / 8 heads x 128: 1350 us against 1262 in turns).  A turn
      // is passed 32 keys before its end, about as long as the passing takes (at
      // the end: 1282; after 64 of 128 keys: 1274; finished blocks of 256 tokens, 16 / 4
      // heads x 64: 75.6, 77.1 and 77.1).
      const int turns = min(c0, c1);
      auto take_turn = [&](int x) {
        if (x >= turns) return true;
        const bool mine = wait(&sh.turn[i][quad], nt ^ (i == 0 ? 1u : 0u), abort_flag);
        nt ^= 1;
        return mine;
      };
      auto pass_turn = [&](int x) {
        if (x < turns && lane == 0) mbar_arrive(&sh.turn[i ^ 1][quad]);
      };
      float m_run = -CUDART_INF_F, l_run = 0.f;
      for (int x = 0; x < c; ++x, ++ns) {
        // P V tiles finished when this tile's P is written: all but this item's first
        // tile's predecessor, which the item before it has waited for
        const uint32_t npv = ns - 1;
        const int t = it.ts + (pair ? x : 2 * x + i);
        if (!wait(&sh.s_full[i], ns & 1, abort_flag)) {
          ok = false;
          break;
        }
        if (ns == 0 && tid == 0) DLM_TRACE_MARK(4);
        // Dh 128: S(x) was finished after P(x-1) V, so O holds every earlier tile and P's
        // columns are free; Dh 64: wait for that (warps without rows as well: they
        // must not announce a P before the last one has been taken)
        if (DH == 64 && x > 0 && !wait(&sh.pv_done[i], npv & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (any) {   // warps without rows leave their lanes of P as they are
          const int left = lim - t * kKeys;
          if (lim_min - t * kKeys < kKeys) {
            // hidden keys: their scores become -inf in tensor memory (few tiles, so
            // the loops below need no mask)
#pragma unroll 1
            for (int y = 0; y < kKeys / 32; ++y) {
              uint32_t raw[32];
              tmem_ld32_nowait(s_col + y * 32, raw);
              tmem_wait_ld();
#pragma unroll
              for (int z = 0; z < 32; ++z)
                if (y * 32 + z >= left) raw[z] = 0xff800000u;
              tmem_st32_u(s_col + y * 32, raw);
            }
            tmem_wait_st();
          }
          // The scores are read twice, for the maximum and for the exponentials,
          // in loops of 32 columns: unrolled over 128 columns in registers the code
          // fell out of the instruction caches, which held up the MMA warp
          float mx = -CUDART_INF_F;
#pragma unroll 1
          for (int y = 0; y < kKeys / 64; ++y) {
            uint32_t r0[32], r1[32];
            tmem_ld32_nowait(s_col + y * 64, r0);
            tmem_ld32_nowait(s_col + y * 64 + 32, r1);
            tmem_wait_ld();
            float m4[4] = {mx, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int z = 0; z < 32; ++z)
              m4[z & 3] = fmax3f(m4[z & 3], __uint_as_float(r0[z]), __uint_as_float(r1[z]));
            mx = fmax3f(m4[0], m4[1], fmaxf(m4[2], m4[3]));
          }
          mx *= p.scale_log2;
          // A row's reference follows its own scores alone.  Lanes that hold no row score
          // whatever lies in their rows of Q and in the slots behind the sequence, and other
          // rows see other keys: a reference shared by the warp would let those decide how
          // this row's P is scaled when it is rounded to bf16.  The vote is only for the
          // rescaling of O, which the warp's loads and stores do together.
          const bool rises = mx > m_run + kRescaleLog2;
          const bool move = __any_sync(0xffffffffu, rises && live);
          const float m_new = rises ? mx : m_run;
          const float base = m_new == -CUDART_INF_F ? 0.f : m_new;   // no key seen yet
          const float alpha = rises ? fast_exp2(m_run - base) : 1.f;
          if (x > 0 && move) {
#pragma unroll 1
            for (int y = 0; y < DH / 32; ++y) {
              float o[32];
              tmem_ld32(o_col + y * 32, o);
#pragma unroll
              for (int z = 0; z < 32; ++z) o[z] *= alpha;
              tmem_st32(o_col + y * 32, o);
            }
          }
          const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), base2 = pack2(-base, -base);
          uint64_t rs[2] = {0, 0};
          // P in the MMA's operand type, two keys a column; the sum keeps float32
          auto exp32 = [&](const uint32_t (&raw)[32], uint32_t (&w)[16]) {
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              float e0, e1;
              const uint64_t x = fma2(
                  pack2(__uint_as_float(raw[2 * z]), __uint_as_float(raw[2 * z + 1])), scale2, base2);
              unpack2(x, e0, e1);
              e0 = fast_exp2(e0);
              e1 = fast_exp2(e1);
              rs[z & 1] = add2(rs[z & 1], pack2(e0, e1));
              w[z] = pack_bf16(e0, e1);
            }
          };
          uint32_t ra[32], rb[32];
          tmem_ld32_nowait(s_col, ra);
          tmem_ld32_nowait(s_col + 32, rb);
          if (!take_turn(x)) {
            ok = false;
            break;
          }
          // 64 keys at a time.  The first half's P is announced when all of S has
          // been read as well: its P V, and what of the next S does not need the
          // second half, run during the second half's exponentials
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t wa[16], wb[16];
            tmem_wait_ld();
            exp32(ra, wa);
            if (h == 0) tmem_ld32_nowait(s_col + 64, ra);
            if (h == 1) pass_turn(x);
            exp32(rb, wb);
            if (h == 0) {
              tmem_ld32_nowait(s_col + 96, rb);
              tmem_wait_ld();
            }
            tmem_st16_u(p_col + h * 32, wa);
            tmem_st16_u(p_col + h * 32 + 16, wb);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[i][h]);
          }
          {
            float s0, s1;
            unpack2(add2(rs[0], rs[1]), s0, s1);
            l_run = l_run * alpha + (s0 + s1);
          }
          m_run = m_new;
        } else {
          if (!take_turn(x)) {
            ok = false;
            break;
          }
          pass_turn(x);
          tc_fence_before();
          __syncwarp();
          if (lane < 2) mbar_arrive(&sh.p_full[i][lane]);
        }
        if (ns == 0 && tid == 0) DLM_TRACE_MARK(5);
      }
      if (!ok) break;
      // the rows' maximum and sum for the writers
      if (!wait(&sh.stat_empty[i], (n & 1) ^ 1, abort_flag)) break;
      sh.stat[i][row] = make_float2(m_run, l_run);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.stat_full[i]);
        mbar_arrive(&sh.d_empty[ds]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort_flag) raise_error(p.err, DLM_ETIMEOUT);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(CUtensorMap* m, void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(api_encode_tiled());
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn != nullptr &&
         fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH>
cudaError_t launch(const PagedAttn& a, int num_sms, cudaStream_t st) {
  static DeviceOnce once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(paged_attn_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<DH>::kBytes);
  });
  if (e != cudaSuccess) return e;
  Params p = make_params(a, num_sms);
  p.npos = kRows / p.G;
  p.positions = 2 * p.npos;
  const cuuint64_t rows = (cuuint64_t)1 << a.c.page_shift;
  const cuuint64_t kd[5] = {64, 8, DH / 64, rows / 8, (cuuint64_t)a.c.n_pages * a.c.Hkv};
  const cuuint64_t ks[4] = {DH * 2, 128, DH * 16, rows * DH * 2};
  const cuuint32_t kb[5] = {64, 8, DH / 64, (cuuint32_t)(rows < kKeys ? rows : kKeys) / 8, 1};
  const cuuint64_t qd[3] = {DH, (cuuint64_t)a.H, (cuuint64_t)a.T};
  const cuuint64_t qst[2] = {DH * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.npos};
  CUtensorMap tmK, tmV, tmQ;
  if (!encode(&tmK, a.c.k, 5, kd, ks, kb) || !encode(&tmV, a.c.v, 5, kd, ks, kb) ||
      !encode(&tmQ, const_cast<void*>(a.q), 3, qd, qst, qb))
    return cudaErrorInvalidValue;
  e = launch_pdl(paged_attn_kernel<DH>, dim3(num_sms), dim3(kThreads), Smem<DH>::kBytes, st, tmK, tmV,
                 tmQ, p);
  if (e != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, DH>(p, num_sms, kSlotRows, st);
}

}  // namespace

size_t paged_attention_work(int Dh, int num_sms) {
  return work_bytes(num_sms, Dh);
}

cudaError_t paged_attention_tc(const PagedAttn& a, int num_sms, cudaStream_t st) {
  return a.c.Dh == 128 ? launch<128>(a, num_sms, st) : launch<64>(a, num_sms, st);
}

}  // namespace dlm
