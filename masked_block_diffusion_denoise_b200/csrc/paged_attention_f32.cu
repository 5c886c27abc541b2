// float32 attention of ragged chunks over a paged KV cache, on the CUDA cores
// (the float32 model; its products would lose half of their bits on the tensor
// cores).
//
// A CTA of 256 threads takes 64 query rows (positions x the G heads of a KV
// head) and walks its key tiles: S = Q K^T and O += P V as register tiles of 4
// rows x (BN / 16) keys or (Dh / 16) columns a thread, four steps of the
// reduction at a time from rows in shared memory (8 16-byte loads for 64 FMAs).
// Q and the K and V tiles come by cp.async, the next tile during this one's
// arithmetic.  Work is cut into equal ranges over all CTAs and joined as in the
// bf16 kernel, so that a few short sequences still spread over the GPU.
//
// All 64 rows are computed, however few hold a query, and every K and V element is
// multiplied with each: 32 FLOP a byte, which caps items of few rows at 1 TB/s (single
// tokens of 61 sequences over 1024..4096 keys, 4 KV heads x 64: 318 us, 1.03 TB/s, with
// 1 and with 4 query heads a KV head; bytes alone 50 us).
//
// Bound by latency for chunks of the float32 model's sizes (4 heads x 64, 9 chunks of up to
// 96 tokens over up to 500 keys, causal, 0.12 GFLOP: 22.9 us a call with the join).  At
// larger ones (700..2000 tokens over up to 4000 keys) it reaches 32 TFLOP/s: eight
// 16-byte loads from shared memory for 64 FMAs a thread.
#include "paged_attn.cuh"

namespace dlm {

namespace {

constexpr int kRows = 64, kThreads = 256, kCtasPerSm = 2;

template <int DH>
struct Shape {
  static constexpr int BN = DH == 128 ? 32 : 64;       // keys per tile
  static constexpr int KN = BN / 16, DN = DH / 16;     // of a thread
  // floats between rows: 4 more than the row, so that 8 rows' 16-byte loads meet
  // 32 different banks
  static constexpr int kLd = DH + 4, kLdP = BN + 4;
  // shared memory, in floats: Q, two K tiles, two V tiles, P
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kRows * kLd;
  static constexpr int kV = kK + 2 * BN * kLd;
  static constexpr int kP = kV + 2 * BN * DH;
  static constexpr int kBytes = (kP + kRows * kLdP) * 4;
};
static_assert(kCtasPerSm * (Shape<128>::kBytes + 2048) <= 227 * 1024 &&
                  kCtasPerSm * (Shape<64>::kBytes + 2048) <= 227 * 1024,
              "two CTAs per SM");

// four floats of shared memory, as two pairs
__device__ __forceinline__ ulonglong2 lds4(const float* p) {
  return *reinterpret_cast<const ulonglong2*>(p);
}

// 16 bytes into shared memory, zeros if !live
__device__ __forceinline__ void copy16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_attn_f32_kernel(const Params p) {
  using SH = Shape<DH>;
  constexpr int BN = SH::BN, KN = SH::KN, DN = SH::DN;
  extern __shared__ __align__(16) float sm[];
  constexpr int kLd = SH::kLd, kLdP = SH::kLdP;
  float* qs = sm + SH::kQ;   // [kRows][kLd]
  float* ks = sm + SH::kK;   // [2][BN][kLd]
  float* vs = sm + SH::kV;   // [2][BN][DH]
  float* ps = sm + SH::kP;   // [kRows][kLdP]
  __shared__ int start[4], stop[4];
  __shared__ longlong2 scan[kThreads / 32];
  __shared__ Item item;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ty = tid >> 4, tx = tid & 15;   // rows 4 ty .., keys tx + 16 j, columns DN tx ..
  pdl_wait_then_release();
  find_range<kThreads>(p, BN, BN, 1, scan, start, stop);
  __syncthreads();
  Walker walk(start, stop);
  const float* kc = (const float*)p.k;
  const float* vc = (const float*)p.v;
  const int page_mask = (1 << p.page_shift) - 1;

  for (;;) {
    if (warp == 0) {
      const Item next = walk.next(p, BN, lane);
      if (lane == 0) item = next;
    }
    __syncthreads();
    const Item it = item;
    if (!it.valid) break;
    const int rows = it.npos * p.G;
    // G > 64: the item's single position in two passes
    for (int r0 = 0; r0 < rows; r0 += kRows) {
      // this thread's rows: what they see
      int lim[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty * 4 + i;
        lim[i] = r < rows ? visible(it.pos0 + div_g(p, r), it.ctx, p.block) : 0;
      }
      __syncthreads();   // the rows before these are done with Q, K, V and P
      // (rows without keys load nothing: nothing waits for such a copy, and it would
      // race with the next item's into the same place)
      const int q_end = it.ts < it.te ? kRows * DH / 4 : 0;
#pragma unroll 4
      for (int x = tid; x < q_end; x += kThreads) {
        const int lr = x / (DH / 4), c = x % (DH / 4) * 4, r = r0 + lr;
        const int pos = div_g(p, r), h = it.g * p.G + r - pos * p.G;
        const bool live = r < rows;
        copy16(qs + lr * kLd + c,
               (const float*)p.q + (live ? (it.row0 + pos) * p.q_stride + (int64_t)h * DH + c : 0), live);
      }
      // K and V of tile t into buffer t & 1; keys behind the sequence are zero
      auto load = [&](int t) {
        float* kd = ks + (t & 1) * BN * kLd;
        float* vd = vs + (t & 1) * BN * DH;
#pragma unroll 4
        for (int x = tid; x < BN * DH / 4; x += kThreads) {
          const int j = x / (DH / 4), c = x % (DH / 4) * 4, k = t * BN + j;
          bool live = k < it.ctx;
          int64_t at = 0;
          if (live) {
            const int page = p.table[(size_t)it.b * p.W + (k >> p.page_shift)];
            live = page >= 0 && page < p.n_pages;
            if (live)
              at = ((((int64_t)page * p.Hkv + it.g) << p.page_shift) + (k & page_mask)) * DH + c;
            else
              raise_error(p.err, DLM_EBOUNDS);
          }
          copy16(kd + j * kLd + c, kc + at, live);
          copy16(vd + j * DH + c, vc + at, live);
        }
        copy_commit();
      };
      if (it.ts < it.te) load(it.ts);
      float m[4], l[4];
      uint64_t acc[4][DN / 2];   // pairs of columns
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DN / 2; ++j) acc[i][j] = 0;
      }
      for (int t = it.ts; t < it.te; ++t) {
        const int k0 = t * BN;
        if (t + 1 < it.te) {
          load(t + 1);
          copy_wait<1>();
        } else {
          copy_wait<0>();
        }
        __syncthreads();
        // S = Q K^T
        // (packed pairs: the even and the odd columns' sums)
        uint64_t s2[4][KN];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < KN; ++j) s2[i][j] = 0;
        const float* kt = ks + (t & 1) * BN * kLd;
        const float* vt = vs + (t & 1) * BN * DH;
#pragma unroll 2
        for (int d = 0; d < DH; d += 4) {
          ulonglong2 b[KN];
#pragma unroll
          for (int j = 0; j < KN; ++j) b[j] = lds4(kt + (tx + 16 * j) * kLd + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const ulonglong2 a = lds4(qs + (ty * 4 + i) * kLd + d);
#pragma unroll
            for (int j = 0; j < KN; ++j) s2[i][j] = fma2(a.y, b[j].y, fma2(a.x, b[j].x, s2[i][j]));
          }
        }
        float s[4][KN];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < KN; ++j) {
            float even, odd;
            unpack2(s2[i][j], even, odd);
            s[i][j] = even + odd;
          }
        // softmax: a row's 16 threads are 16 lanes of a warp
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int j = 0; j < KN; ++j) {
            s[i][j] = k0 + tx + 16 * j < lim[i] ? s[i][j] * p.scale_log2 : -CUDART_INF_F;
            mx = fmaxf(mx, s[i][j]);
          }
#pragma unroll
          for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          const float m_new = fmaxf(m[i], mx);
          const float base = m_new == -CUDART_INF_F ? 0.f : m_new;   // no key seen yet
          const float alpha = fast_exp2(m[i] - base);
          m[i] = m_new;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < KN; ++j) {
            s[i][j] = fast_exp2(s[i][j] - base);
            sum += s[i][j];
          }
          l[i] = l[i] * alpha + sum;   // this thread's keys; added up at the end
#pragma unroll
          for (int j = 0; j < DN / 2; ++j) acc[i][j] = mul2(acc[i][j], pack2(alpha, alpha));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < KN; ++j) ps[(ty * 4 + i) * kLdP + tx + 16 * j] = s[i][j];
        __syncwarp();   // a row's P is written and read by one half-warp
        // O += P V; in tiles with hidden keys a row takes nothing from the V of those
        // (0 x infinity would be NaN).  Asked of the key, not of its probability: a seen
        // key's may underflow to 0, and its V still counts if it is not finite
        auto pv = [&](auto hidden) {
#pragma unroll 2
          for (int k = 0; k < BN; k += 4) {
            uint64_t b[4][DN / 2];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float* src = vt + (k + y) * DH + tx * DN;
              if constexpr (DN == 2) {
                b[y][0] = *reinterpret_cast<const uint64_t*>(src);
              } else {
#pragma unroll
                for (int j = 0; j < DN / 2; j += 2) {
                  const ulonglong2 v = lds4(src + 2 * j);
                  b[y][j] = v.x;
                  b[y][j + 1] = v.y;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 a = *reinterpret_cast<const float4*>(ps + (ty * 4 + i) * kLdP + k);
              const float w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
              for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int j = 0; j < DN / 2; ++j)
                  acc[i][j] = fma2(pack2(w[y], w[y]),
                                   decltype(hidden)::value && k0 + k + y >= lim[i] ? 0ull : b[y][j], acc[i][j]);
            }
          }
        };
        if (k0 + BN > it.fix)
          pv(std::true_type{});
        else
          pv(std::false_type{});
        __syncthreads();   // this buffer is loaded again
      }
      // results
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        const int r = r0 + ty * 4 + i;
        if (r >= rows) continue;
        const int pos = div_g(p, r), h = it.g * p.G + r - pos * p.G;
        const int64_t grow = (int64_t)it.row0 + pos;
        const size_t slot = (size_t)blockIdx.x * 2 + it.slot;
        const float inv = it.whole ? inverse(l[i], lim[i] > 0) : 1.f;
        float* dst = (float*)p.o + grow * p.o_stride + (int64_t)h * DH;
#pragma unroll
        for (int j = 0; j < DN / 2; ++j) {
          const int col = tx * DN + 2 * j;
          *reinterpret_cast<uint64_t*>(it.whole ? dst + col : p.part + part_at<float, DH>(slot, r, col)) =
              mul2(acc[i][j], pack2(inv, inv));
        }
        if (tx == 0) {
          if (!it.whole)
            p.ml[slot * kSlotRows + r] = make_float2(m[i], l[i]);
          else if (p.lse != nullptr)
            p.lse[(size_t)grow * p.H + h] =
                l[i] == 0.f ? -CUDART_INF_F : (m[i] + log2f(l[i])) * 0.69314718055994531f;
        }
      }
    }
    __syncthreads();   // `item` has been read
  }
  if (tid == 0) p.meta[blockIdx.x] = walk.meta;
}

template <int DH>
cudaError_t launch(const PagedAttn& a, int num_sms, cudaStream_t st) {
  static DeviceOnce once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(paged_attn_f32_kernel<DH>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<DH>::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int ctas = num_sms * kCtasPerSm;
  Params p = make_params(a, ctas);
  p.npos = p.G < kRows ? kRows / p.G : 1;
  p.positions = p.npos;
  e = launch_pdl(paged_attn_f32_kernel<DH>, dim3(ctas), dim3(kThreads), Shape<DH>::kBytes, st, p);
  if (e != cudaSuccess) return e;
  return launch_join<float, DH>(p, ctas, p.npos * p.G, st);
}

}  // namespace

size_t paged_attention_f32_work(int Dh, int num_sms) {
  return work_bytes(num_sms * kCtasPerSm, Dh);
}

cudaError_t paged_attention_f32(const PagedAttn& a, int num_sms, cudaStream_t st) {
  if (a.c.Dh == 32) return launch<32>(a, num_sms, st);
  return a.c.Dh == 64 ? launch<64>(a, num_sms, st) : launch<128>(a, num_sms, st);
}

}  // namespace dlm
