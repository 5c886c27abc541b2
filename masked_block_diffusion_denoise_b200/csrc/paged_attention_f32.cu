// float32 attention of ragged chunks over a paged KV cache, on the CUDA cores
// (the float32 model; its products would lose half of their bits on the tensor
// cores).
//
// A CTA of 128 threads takes 64 query rows (positions x the G heads of a KV
// head) and walks its key tiles: S = Q K^T and O += P V as register tiles of 8
// rows x (BN / 16) keys or (Dh / 16) columns a thread, operands by float4 from
// shared memory (Q, K, P with the reduction index outermost).  Two or three CTAs
// per SM hide each other's loads.  Work is cut into equal ranges over all CTAs
// and joined as in the bf16 kernel, so that a few short sequences still spread
// over the GPU.  Bound by the FMA pipe and shared memory.
#include "paged_attn.cuh"

namespace dlm {

namespace {

constexpr int kRows = 64, kThreads = 128;
constexpr int kStride = kRows + 4;   // floats between reduction steps of Q and P

template <int DH>
struct Shape {
  static constexpr int BN = DH == 128 ? 32 : 64;       // keys per tile
  static constexpr int KN = BN / 16, DN = DH / 16;     // of a thread
  static constexpr int kCtasPerSm = DH == 128 ? 2 : 3;
  // shared memory, in floats
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + DH * kStride;
  static constexpr int kV = kK + DH * (BN + 4);
  static constexpr int kP = kV + BN * DH;
  static constexpr int kBytes = (kP + BN * kStride) * 4;
};

// N consecutive floats of shared memory
template <int N>
__device__ __forceinline__ void lds(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads) paged_attn_f32_kernel(const Params p) {
  using SH = Shape<DH>;
  constexpr int BN = SH::BN, KN = SH::KN, DN = SH::DN;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm + SH::kQ;   // [DH][kStride]
  float* ks = sm + SH::kK;   // [DH][BN + 4]
  float* vs = sm + SH::kV;   // [BN][DH]
  float* ps = sm + SH::kP;   // [BN][kStride]
  __shared__ int start[4], stop[4];
  __shared__ long long scan[kThreads / 32];
  __shared__ Item item;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ty = tid >> 4, tx = tid & 15;   // rows 8 ty .., keys KN tx .., columns DN tx ..
  find_range<kThreads>(p, BN, BN, 2 * BN, scan, start, stop);
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
      int lim[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + ty * 8 + i;
        lim[i] = r < rows ? visible(it.pos0 + r / p.G, it.ctx, p.block) : 0;
      }
      __syncthreads();
      // Q, transposed: a lane's row, 4 columns at a time
      for (int x = warp; x < DH / 4 * (kRows / 32); x += kThreads / 32) {
        const int lr = (x % (kRows / 32)) * 32 + lane, c = x / (kRows / 32) * 4;
        const int r = r0 + lr;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
          const int pos = r / p.G, h = it.g * p.G + r - pos * p.G;
          v = __ldg(reinterpret_cast<const float4*>((const float*)p.q + (it.row0 + pos) * p.q_stride +
                                                    (int64_t)h * DH + c));
        }
        qs[(c + 0) * kStride + lr] = v.x;
        qs[(c + 1) * kStride + lr] = v.y;
        qs[(c + 2) * kStride + lr] = v.z;
        qs[(c + 3) * kStride + lr] = v.w;
      }
      float m[8], l[8], acc[8][DN];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DN; ++j) acc[i][j] = 0.f;
      }
      for (int t = it.ts; t < it.te; ++t) {
        const int k0 = t * BN;
        __syncthreads();   // the previous tile is done with
        auto row_of = [&](int j) -> int64_t {   // of key k0 + j in the cache, or -1
          const int k = k0 + j;
          if (k >= it.ctx) return -1;
          const int page = __ldg(p.table + (size_t)it.b * p.W + (k >> p.page_shift));
          if (page < 0 || page >= p.n_pages) {
            raise_error(p.err, DLM_EBOUNDS);
            return -1;
          }
          return (((int64_t)page * p.Hkv + it.g) << p.page_shift) + (k & page_mask);
        };
        {
          // K, transposed (a lane's key); keys behind the sequence are zero
          constexpr int kParts = kThreads / BN;
          const int j = tid % BN;
          const int64_t row = row_of(j);
          const float4* src = reinterpret_cast<const float4*>(kc + row * DH);
#pragma unroll 8
          for (int c = tid / BN; c < DH / 4; c += kParts) {
            const float4 v = row >= 0 ? __ldg(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            ks[(c * 4 + 0) * (BN + 4) + j] = v.x;
            ks[(c * 4 + 1) * (BN + 4) + j] = v.y;
            ks[(c * 4 + 2) * (BN + 4) + j] = v.z;
            ks[(c * 4 + 3) * (BN + 4) + j] = v.w;
          }
        }
#pragma unroll 4
        for (int x = tid; x < BN * DH / 4; x += kThreads) {
          const int64_t row = row_of(x / (DH / 4));
          reinterpret_cast<float4*>(vs)[x] =
              row >= 0 ? __ldg(reinterpret_cast<const float4*>(vc + row * DH) + x % (DH / 4))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        // S = Q K^T
        float s[8][KN];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < KN; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < DH; ++d) {
          float a[8], b[KN];
          lds<8>(qs + d * kStride + ty * 8, a);
          lds<KN>(ks + d * (BN + 4) + tx * KN, b);
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < KN; ++j) s[i][j] = fmaf(a[i], b[j], s[i][j]);
        }
        // softmax: a row's 16 threads are 16 lanes of a warp
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int j = 0; j < KN; ++j) {
            s[i][j] = k0 + tx * KN + j < lim[i] ? s[i][j] * p.scale_log2 : -CUDART_INF_F;
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
          for (int j = 0; j < DN; ++j) acc[i][j] *= alpha;
        }
#pragma unroll
        for (int j = 0; j < KN; ++j) {
          float* dst = ps + (tx * KN + j) * kStride + ty * 8;
          *reinterpret_cast<float4*>(dst) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(s[4][j], s[5][j], s[6][j], s[7][j]);
        }
        __syncthreads();
        // O += P V; in tiles with hidden keys a probability of 0 takes nothing
        // from V (0 x infinity would be NaN)
        auto pv = [&](auto hidden) {
#pragma unroll 4
          for (int k = 0; k < BN; ++k) {
            float a[8], b[DN];
            lds<8>(ps + k * kStride + ty * 8, a);
            lds<DN>(vs + k * DH + tx * DN, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < DN; ++j)
                acc[i][j] = fmaf(a[i], decltype(hidden)::value && a[i] == 0.f ? 0.f : b[j], acc[i][j]);
          }
        };
        if (k0 + BN > it.fix)
          pv(std::true_type{});
        else
          pv(std::false_type{});
      }
      // results
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        const int r = r0 + ty * 8 + i;
        if (r >= rows) continue;
        const int pos = r / p.G, h = it.g * p.G + r - pos * p.G;
        const int64_t grow = (int64_t)it.row0 + pos;
        const size_t prow = ((size_t)blockIdx.x * 2 + it.slot) * kSlotRows + r;
        const float inv = !it.whole ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
        float* dst = it.whole ? (float*)p.o + grow * p.o_stride + (int64_t)h * DH : p.part + prow * DH;
#pragma unroll
        for (int j = 0; j < DN; j += 2)
          *reinterpret_cast<float2*>(dst + tx * DN + j) =
              make_float2(acc[i][j] * inv, acc[i][j + 1] * inv);
        if (tx == 0) {
          if (!it.whole)
            p.ml[prow] = make_float2(m[i], l[i]);
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
  const int ctas = num_sms * Shape<DH>::kCtasPerSm;
  Params p = make_params(a, ctas);
  p.npos = p.G < kRows ? kRows / p.G : 1;
  p.positions = p.npos;
  paged_attn_f32_kernel<DH><<<ctas, kThreads, Shape<DH>::kBytes, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<float, DH>(p, ctas, p.npos * p.G, st);
}

}  // namespace

size_t paged_attention_f32_work(int Dh, int num_sms) {
  return work_bytes(num_sms * (Dh == 128 ? Shape<128>::kCtasPerSm : Shape<64>::kCtasPerSm), Dh);
}

cudaError_t paged_attention_f32(const PagedAttn& a, int num_sms, cudaStream_t st) {
  if (a.c.Dh == 32) return launch<32>(a, num_sms, st);
  return a.c.Dh == 64 ? launch<64>(a, num_sms, st) : launch<128>(a, num_sms, st);
}

}  // namespace dlm
