// kv_append.hip -- new keys and values into a paged cache, the keys rotated on the way, and
// the new queries rotated with them (kv_append of include/attn.h).
//
// Mathematics: the rotation of rope_qk.h, value for value: angle fp32(p / pos_scale) *
// inv_freq[j], correctly rounded fp32 cos and sin (cr_sincos.h), and each output as a 2x2
// determinant by Kahan's FMA scheme (Jeannerod, Louvet, Muller, Math. Comp. 82 (2013)), within
// 2 fp32 ulps before the one rounding to storage.
//
// What bounds it: memory; every element is read once and written once. One workgroup per
// token: its first D/2 lanes evaluate the token's cos/sin once for all heads, into LDS,
// while the loads of its first chunk pairs are in flight. Rows are moved as pairs of chunks
// (VEC elements of either half row), V's without a rotation. Measured, bf16, 32 + 8 heads of
// 128: 4001 tokens of each of four prompts 72 us at best and 76 in the middle of many launches, 5.5
// and 5.2 TB/s (a large copy moves 5.0); one token of each of 64 sequences 5 us, latency.
#include "attn_common.h"
#include "cr_sincos.h"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxHalf = 256;
constexpr int kUnroll = 4;

struct AppendParams {
  const void* q;
  void* q_out;
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* kv_lens;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  int64_t page_stride, slot_stride, head_stride, table_stride;
  int32_t T, num_seqs, Hq, Hkv, D, num_pages, page_size, max_pages;
  float pos_scale;
  Div31 by_page, by_pairs;
  float inv_freq[kMaxHalf];
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Chunk {
  T v[VEC];
};

template <typename T>
__device__ inline T narrow(float x) { return (T)x; }

// Sequence of token t: the last s with cu[s] <= t, or -1 (also behind the last sequence).
__device__ inline int32_t find_sequence(const int32_t* __restrict__ cu, int32_t num_seqs, int32_t t) {
  if (num_seqs == 0) return -1;
  int32_t first = 0, count = num_seqs + 1;
  while (count > 0) {
    const int32_t step = count >> 1;
    if (cu[first + step] <= t) {
      first += step + 1;
      count -= step + 1;
    } else {
      count = step;
    }
  }
  return first - 1 < num_seqs ? first - 1 : -1;
}

template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(const AppendParams p) {
  using C = Chunk<T, VEC>;
  __shared__ float cs[kMaxHalf], sn[kMaxHalf];
  const int32_t t = blockIdx.x;
  const int32_t half = p.D >> 1, pairs = half / VEC;

  const int32_t s = find_sequence(p.cu, p.num_seqs, t);
  int64_t pos = -1;
  int64_t row = -1;  // the token's row of the cache, in elements from its base
  if (s >= 0) {
    pos = (int64_t)p.kv_lens[s] - min(p.cu[s + 1], p.T) + t;  // as paged_plan reads it
    if (pos >= 0 && pos < INT32_MAX) {
      const uint32_t block = div31((uint32_t)pos, p.by_page);
      if (block < (uint32_t)p.max_pages) {
        const int32_t page = p.table[s * p.table_stride + block];
        if (page >= 0 && page < p.num_pages)
          row = page * p.page_stride + (int64_t)((uint32_t)pos - block * p.page_size) * p.slot_stride;
      }
    }
  }
  const bool turn = pos >= 0 && pos < INT32_MAX;
  const bool move_q = p.q != nullptr && (turn || p.q != p.q_out);

  // items: chunk pairs of the rows of Q, of K, of V
  const int32_t nq = p.Hq * pairs, nk = p.Hkv * pairs;
  const int32_t begin = move_q ? 0 : nq;
  const int32_t end = row >= 0 ? nq + 2 * nk : nq;
  if (begin >= end) return;
  const T* q = static_cast<const T*>(p.q) + (int64_t)t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + (int64_t)t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + (int64_t)t * p.v_stride;
  T* q_out = static_cast<T*>(p.q_out) + (int64_t)t * p.q_out_stride;
  T* kc = static_cast<T*>(p.k_cache) + row;
  T* vc = static_cast<T*>(p.v_cache) + row;

  for (int32_t i0 = begin; i0 < end; i0 += kUnroll * kThreads) {
    C lo[kUnroll], hi[kUnroll];
    int32_t head[kUnroll], chunk[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t i = i0 + u * kThreads + threadIdx.x;
      if (i < end) {
        const T* src = i < nq ? q : i < nq + nk ? k : v;
        const int32_t of = i < nq ? i : i < nq + nk ? i - nq : i - nq - nk;
        head[u] = div31(of, p.by_pairs);
        chunk[u] = of - head[u] * pairs;
        src += (int64_t)head[u] * p.D + chunk[u] * VEC;
        lo[u] = *reinterpret_cast<const C*>(src);
        hi[u] = *reinterpret_cast<const C*>(src + half);
      }
    }
    if (i0 == begin) {  // the same for the whole workgroup
      if (turn) {
        const float fp = (float)(int32_t)pos;
        const float scaled = p.pos_scale == 1.0f ? fp : __fdiv_rn(fp, p.pos_scale);
        for (int32_t j = threadIdx.x; j < half; j += kThreads) {
          float sine, cosine;
          rope_trig::sincos_f32_cr(__fmul_rn(scaled, p.inv_freq[j]), sine, cosine);
          cs[j] = cosine;
          sn[j] = sine;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t i = i0 + u * kThreads + threadIdx.x;
      if (i < end) {
        if (turn && i < nq + nk) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float x1 = (float)lo[u].v[e], x2 = (float)hi[u].v[e];
            const float c = cs[chunk[u] * VEC + e], z = sn[chunk[u] * VEC + e];
            const float w1 = x2 * z;
            const float e1 = __builtin_fmaf(-x2, z, w1);
            const float w2 = x1 * z;
            const float e2 = __builtin_fmaf(x1, z, -w2);
            lo[u].v[e] = narrow<T>(__builtin_fmaf(x1, c, -w1) + e1);
            hi[u].v[e] = narrow<T>(__builtin_fmaf(x2, c, w2) + e2);
          }
        }
        T* dst = i < nq ? q_out + (int64_t)head[u] * p.D
                        : (i < nq + nk ? kc : vc) + (int64_t)head[u] * p.head_stride;
        dst += chunk[u] * VEC;
        *reinterpret_cast<C*>(dst) = lo[u];
        *reinterpret_cast<C*>(dst + half) = hi[u];
      }
    }
  }
}

template <typename T>
int32_t launch(const AppendParams& p, int32_t bytes, hipStream_t s) {
  const dim3 grid((unsigned)p.T), block(kThreads);
  switch (bytes / (int32_t)sizeof(T)) {
    case 1: hipLaunchKernelGGL((kv_append_kernel<T, 1>), grid, block, 0, s, p); break;
    case 2: hipLaunchKernelGGL((kv_append_kernel<T, 2>), grid, block, 0, s, p); break;
    case 4: hipLaunchKernelGGL((kv_append_kernel<T, 4>), grid, block, 0, s, p); break;
    default:
      if constexpr (sizeof(T) == 2)
        hipLaunchKernelGGL((kv_append_kernel<T, 8>), grid, block, 0, s, p);
      else
        return ROPE_EINVAL;
  }
  return launched();
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" int32_t kv_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                             void* v_cache, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                             int64_t q_stride, int64_t q_out_stride, int64_t k_stride,
                             int64_t v_stride, int32_t num_pages, int32_t page_size,
                             int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                             const int32_t* block_table, int32_t max_pages, int64_t table_stride,
                             const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* kv_lens,
                             double theta, double pos_scale, int32_t dtype, void* stream) {
  if (dtype != ROPE_F32 && dtype != ROPE_BF16 && dtype != ROPE_F16) return ROPE_EUNSUPPORTED;
  if (T < 0 || T > kMaxBlocks || Hq < 0 || Hq > kMaxHeads || Hkv < 1 || Hkv > kMaxHeads)
    return ROPE_EINVAL;
  AppendParams p;
  if (D < 2 || D > 2 * kMaxHalf || rope_inv_freq(theta, D, p.inv_freq) != ROPE_OK) return ROPE_EINVAL;
  p.pos_scale = (float)pos_scale;
  if (!(p.pos_scale >= 1.0f) || p.pos_scale > 3e38f) return ROPE_EINVAL;
  if (num_seqs < 0 || num_seqs > (1 << 24) || num_pages < 0 || page_size < 1 || max_pages < 0)
    return ROPE_EINVAL;
  const int64_t dense_q = (int64_t)Hq * D, dense_k = (int64_t)Hkv * D, most = (int64_t)1 << 40;
  p.q_stride = q_stride == 0 ? dense_q : q_stride;
  p.q_out_stride = q_out_stride == 0 ? dense_q : q_out_stride;
  p.k_stride = k_stride == 0 ? dense_k : k_stride;
  p.v_stride = v_stride == 0 ? dense_k : v_stride;
  if (p.q_stride < dense_q || p.q_out_stride < dense_q || p.k_stride < dense_k ||
      p.v_stride < dense_k || p.q_stride > most || p.q_out_stride > most || p.k_stride > most ||
      p.v_stride > most)
    return ROPE_EINVAL;
  if (page_stride < 0 || slot_stride < 0 || head_stride < 0 || page_stride > most ||
      slot_stride > most || head_stride > most || table_stride < 0 || table_stride > most)
    return ROPE_EINVAL;
  if (T == 0) return ROPE_OK;
  if (num_seqs > 0 && (cu_seqlens == nullptr || kv_lens == nullptr)) return ROPE_EINVAL;
  if (max_pages > 0 && num_seqs > 0 && block_table == nullptr) return ROPE_EINVAL;
  if (k == nullptr || v == nullptr || (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)))
    return ROPE_EINVAL;
  if (Hq > 0 && q != nullptr && q_out == nullptr) return ROPE_EINVAL;
  const bool has_q = Hq > 0 && q != nullptr;
  if (has_q && q == q_out && p.q_stride != p.q_out_stride) return ROPE_EINVAL;

  // the widest chunk that divides a half row and keeps every access aligned
  const int32_t size = dtype == ROPE_F32 ? 4 : 2;
  int32_t bytes = 16;
  const int64_t of[] = {(int64_t)D / 2 * size, p.k_stride * size, p.v_stride * size,
                        page_stride * size, slot_stride * size, head_stride * size,
                        (int64_t)(uintptr_t)k, (int64_t)(uintptr_t)v, (int64_t)(uintptr_t)k_cache,
                        (int64_t)(uintptr_t)v_cache, has_q ? p.q_stride * size : 0,
                        has_q ? p.q_out_stride * size : 0, has_q ? (int64_t)(uintptr_t)q : 0,
                        has_q ? (int64_t)(uintptr_t)q_out : 0};
  for (const int64_t x : of)
    while (bytes > size && x % bytes != 0) bytes >>= 1;

  p.q = has_q ? q : nullptr;
  p.q_out = has_q ? q_out : nullptr;
  p.k = k;
  p.v = v;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.table = block_table;
  p.cu = cu_seqlens;
  p.kv_lens = kv_lens;
  p.page_stride = page_stride;
  p.slot_stride = slot_stride;
  p.head_stride = head_stride;
  p.table_stride = table_stride;
  p.T = (int32_t)T;
  p.num_seqs = num_seqs;
  p.Hq = has_q ? Hq : 0;
  p.Hkv = Hkv;
  p.D = D;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.by_page = make_div31(page_size);
  p.by_pairs = make_div31(D / 2 * size / bytes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (dtype) {
    case ROPE_F32: return launch<float>(p, bytes, s);
    case ROPE_BF16: return launch<__bf16>(p, bytes, s);
    default: return launch<_Float16>(p, bytes, s);
  }
}
