// rope_axes.hip -- the rotary embedding by positions with several axes (include/rope_axes.h): of
// queries and keys, either way round, and on the way into the cache rows of a slot map.
//
// Mathematics: as in kv_append.hip, with the angle of frequency j from the position on its axis.
//
// What bounds it: memory; every element is read once and written once. A workgroup takes `group`
// consecutive tokens, as many as give each of its threads two or four pairs of chunks (fewer
// where that would leave CUs without work): the loads of all of them are begun, cos and sin of the
// tokens' frequencies are evaluated into LDS while they are on the way, and the pairs are rotated
// and written, past the caches (non-temporal). Loads go past them too where a half row is whole
// 128-byte lines, which no other chunk then needs again. Measured, GPU time at bf16 and 32 + 8 heads of
// 128, 10814 tokens: 52 us through the caches, 43 with such stores, 40.5 with loads too, which is 5.5
// TB/s (a large copy moves 5.1); 16 + 16 heads of 96: 36.5, 26.6, and 30.8, for lines are fetched
// twice. 16004 tokens of 32 + 8 heads into the cache: 87, 74, 70 us. Workgroups of 64, 256 or 512 threads
// were up to 25 % slower on some of twelve such shapes and nowhere faster than 10 %. Where there are more
// tokens than a dispatch has workgroups, each takes as many as that needs, whatever its work.
#include "attn_common.h"
#include "cr_sincos.h"
#include "storage.h"
#include "../../include/rope_axes.h"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxHalf = 256;
// Chunk pairs of a thread whose loads are in flight together. Two where the rotation alone moves 16-byte
// chunks that share lines (16 + 16 heads of 80, 8641 tokens: 18.1 us, and 20.1 with four; 32 + 8 heads of 32: 13.0
// and 15.5; of 96: 24.6 and 26.6; of 64: the same), four elsewhere (heads of 72, 8-byte chunks: 13.0, and 16.8 with
// two; into the cache, heads of 64: 39.9 and 44.9).
constexpr int unroll(int chunk_bytes, bool slots, bool lines) {
  return chunk_bytes == 16 && !slots && !lines ? 2 : 4;
}
constexpr int kMostTokens = 16;        // of a workgroup
constexpr int kTableFloats = 2048;     // of cos, and of sin: 16 KB of LDS
constexpr int64_t kFewest = 1024;      // workgroups, where there are tokens for them
constexpr int64_t kMostGroups = 0xffffffff / kThreads;  // of a dispatch

struct AxesParams {
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  const void* v;        // with slots
  void* v_out;
  const int64_t* slots; // or NULL
  const int32_t* ids;
  int64_t q_stride, q_out_stride, k_stride, k_out_stride, v_stride, ids_stride;
  int64_t page_stride, slot_stride, head_stride, num_slots;
  int32_t T, Hq, Hkv, D, axes, page_size, group;
  float pos_scale, sign;
  Div31 by_page, by_pairs, by_token, by_half;
  uint32_t axis[kMaxHalf / 16];  // of each frequency, two bits
  float inv_freq[kMaxHalf];
};

template <typename T, int VEC, bool SLOTS, bool LINES>
__global__ __launch_bounds__(kThreads) void rope_axes_kernel(const AxesParams p) {
  using C = storage::Chunk<T, VEC>;
  constexpr int kUnroll = unroll(VEC * sizeof(T), SLOTS, LINES);
  __shared__ float cs[kTableFloats], sn[kTableFloats];
  __shared__ int64_t row_of[kMostTokens];  // of the cache, in elements; < 0: none
  __shared__ uint8_t turns[kMostTokens];
  const int32_t t0 = blockIdx.x * p.group;
  const int32_t tokens = min(p.group, p.T - t0);
  const int32_t half = p.D >> 1, pairs = half / VEC;
  if ((int32_t)threadIdx.x < tokens) {
    const int32_t t = t0 + threadIdx.x;
    bool turn = true;
    for (int32_t a = 0; a < p.axes; ++a) turn &= p.ids[a * p.ids_stride + t] >= 0;
    turns[threadIdx.x] = turn;
    if constexpr (SLOTS) {
      const int64_t slot = p.slots[t];
      int64_t row = -1;
      if (slot >= 0 && slot < p.num_slots) {
        const int64_t page = slot <= INT32_MAX ? (int64_t)div31((uint32_t)slot, p.by_page) : slot / p.page_size;
        row = page * p.page_stride + (slot - page * p.page_size) * p.slot_stride;
      }
      row_of[threadIdx.x] = row;
    }
  }

  // items: chunk pairs of the rows of Q, of K, of V of each token
  const int32_t nq = p.Hq * pairs, nk = p.Hkv * pairs;
  const int32_t per_token = nq + (SLOTS ? 2 : 1) * nk, end = tokens * per_token;
  for (int32_t i0 = 0; i0 < end; i0 += kUnroll * kThreads) {
    C lo[kUnroll], hi[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t i = i0 + u * kThreads + threadIdx.x;
      if (i < end) {
        const int32_t y = div31(i, p.by_token), of = i - y * per_token;
        const bool is_q = of < nq, is_v = SLOTS && of >= nq + nk;
        const int32_t at = is_q ? of : is_v ? of - nq - nk : of - nq;
        const int32_t h = div31(at, p.by_pairs), c = at - h * pairs;
        const T* src = static_cast<const T*>(is_q ? p.q : is_v ? p.v : p.k) +
                       (int64_t)(t0 + y) * (is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride) +
                       ((int64_t)h * p.D + c * VEC);
        if constexpr (LINES) {
          lo[u] = storage::load_chunk<T, VEC>(src);
          hi[u] = storage::load_chunk<T, VEC>(src + half);
        } else {
          lo[u] = *reinterpret_cast<const C*>(src);
          hi[u] = *reinterpret_cast<const C*>(src + half);
        }
      }
    }
    if (i0 == 0) {  // the same for the whole workgroup
      for (int32_t x = threadIdx.x; x < tokens * half; x += kThreads) {
        const int32_t y = div31(x, p.by_half), j = x - y * half;
        const int32_t axis = p.axis[j >> 4] >> (2 * (j & 15)) & 3;
        const float fp = (float)p.ids[axis * p.ids_stride + t0 + y];
        const float scaled = p.pos_scale == 1.0f ? fp : __fdiv_rn(fp, p.pos_scale);
        float sine, cosine;
        rope_trig::sincos_f32_cr(__fmul_rn(scaled, p.inv_freq[j]), sine, cosine);
        cs[x] = cosine;
        sn[x] = sine * p.sign;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t i = i0 + u * kThreads + threadIdx.x;
      if (i < end) {
        const int32_t y = div31(i, p.by_token), of = i - y * per_token;
        const bool is_q = of < nq, is_v = SLOTS && of >= nq + nk;
        const int32_t at = is_q ? of : is_v ? of - nq - nk : of - nq;
        const int32_t h = div31(at, p.by_pairs), c = at - h * pairs;
        T* to;
        bool write = true;
        if (SLOTS && !is_q) {
          write = row_of[y] >= 0;
          to = static_cast<T*>(is_v ? p.v_out : p.k_out) + row_of[y] + (int64_t)h * p.head_stride;
        } else {
          to = static_cast<T*>(is_q ? p.q_out : p.k_out) +
               (int64_t)(t0 + y) * (is_q ? p.q_out_stride : p.k_out_stride) + (int64_t)h * p.D;
        }
        to += c * VEC;
        if (turns[y] && !is_v) {
          const int32_t x = y * half + c * VEC;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float x1 = (float)lo[u].v[e], x2 = (float)hi[u].v[e];
            const float co = cs[x + e], si = sn[x + e];
            const float w1 = x2 * si;
            const float e1 = __builtin_fmaf(-x2, si, w1);
            const float w2 = x1 * si;
            const float e2 = __builtin_fmaf(x1, si, -w2);
            lo[u].v[e] = (T)(__builtin_fmaf(x1, co, -w1) + e1);
            hi[u].v[e] = (T)(__builtin_fmaf(x2, co, w2) + e2);
          }
        }
        if (write) {
          storage::store_chunk<T, VEC>(to, lo[u]);
          storage::store_chunk<T, VEC>(to + half, hi[u]);
        }
      }
    }
  }
}

inline bool whole_lines(int32_t D, int32_t size) { return D / 2 * size % 128 == 0; }

template <typename T, bool SLOTS>
int32_t launch(const AxesParams& p, int32_t bytes, hipStream_t s) {
  const dim3 grid((unsigned)((p.T + (int64_t)p.group - 1) / p.group)), block(kThreads);
  switch (bytes / (int32_t)sizeof(T)) {
    case 1: hipLaunchKernelGGL((rope_axes_kernel<T, 1, SLOTS, false>), grid, block, 0, s, p); break;
    case 2: hipLaunchKernelGGL((rope_axes_kernel<T, 2, SLOTS, false>), grid, block, 0, s, p); break;
    case 16 / sizeof(T):
      if (whole_lines(p.D, sizeof(T)))
        hipLaunchKernelGGL((rope_axes_kernel<T, 16 / sizeof(T), SLOTS, true>), grid, block, 0, s, p);
      else
        hipLaunchKernelGGL((rope_axes_kernel<T, 16 / sizeof(T), SLOTS, false>), grid, block, 0, s, p);
      break;
    default:
      if constexpr (sizeof(T) == 2)  // 8 bytes
        hipLaunchKernelGGL((rope_axes_kernel<T, 4, SLOTS, false>), grid, block, 0, s, p);
      else
        return ROPE_EINVAL;
  }
  return launched();
}

template <bool SLOTS>
int32_t launch_typed(const AxesParams& p, int32_t bytes, int32_t dtype, hipStream_t s) {
  switch (dtype) {
    case ROPE_F32: return launch<float, SLOTS>(p, bytes, s);
    case ROPE_BF16: return launch<__bf16, SLOTS>(p, bytes, s);
    default: return launch<_Float16, SLOTS>(p, bytes, s);
  }
}

// Axes and inverse frequencies of the D/2 frequencies; false for arguments that give none.
bool set_frequencies(AxesParams& p, int32_t D, const int32_t* sections, int32_t axes, int32_t layout,
                     double theta) {
  if (D < 2 || D > 2 * kMaxHalf || D % 2 != 0 || sections == nullptr || axes < 1 || axes > ROPE_AXES_MOST)
    return false;
  const int32_t half = D / 2;
  int64_t sum = 0;
  for (int32_t a = 0; a < axes; ++a) {
    if (sections[a] < 0 || sections[a] > half) return false;
    sum += sections[a];
  }
  if (sum != half) return false;
  if (rope_inv_freq(theta, D, p.inv_freq) != ROPE_OK) return false;
  uint8_t axis[kMaxHalf];
  if (layout == ROPE_AXES_INTERLEAVED) {
    for (int32_t a = 1; a < axes; ++a)
      if (sections[a] > 0 && axes * (sections[a] - 1) + a >= half) return false;
    for (int32_t j = 0; j < half; ++j) axis[j] = j < axes * sections[j % axes] ? j % axes : 0;
  } else if (layout == ROPE_AXES_SECTIONS || layout == ROPE_AXES_SEPARATE) {
    int32_t j = 0;
    for (int32_t a = 0; a < axes; ++a) {
      // theta^(-i / n) is theta^(-2 i / (2 n)), the ladder of a head of 2 n
      if (layout == ROPE_AXES_SEPARATE && sections[a] > 0 &&
          rope_inv_freq(theta, 2 * sections[a], p.inv_freq + j) != ROPE_OK)
        return false;
      for (int32_t i = 0; i < sections[a]; ++i) axis[j++] = (uint8_t)a;
    }
  } else {
    return false;
  }
  for (uint32_t& w : p.axis) w = 0;
  for (int32_t j = 0; j < half; ++j) p.axis[j >> 4] |= (uint32_t)axis[j] << (2 * (j & 15));
  return true;
}

bool stride_of(int64_t stride, int64_t dense, int64_t* out) {
  *out = stride == 0 ? dense : stride;
  return *out >= dense && *out <= (int64_t)1 << 40;
}

// Chunk size, tokens of a workgroup, divisions; `of`: what bounds the width of accesses, in bytes.
template <size_t N>
int32_t set_geometry(AxesParams& p, int32_t size, bool slots, const int64_t (&of)[N]) {
  int32_t bytes = 16;
  for (const int64_t x : of)
    while (bytes > size && x % bytes != 0) bytes >>= 1;
  const int32_t half = p.D / 2, pairs = half * size / bytes;
  const int32_t per_token = (p.Hq + (slots ? 2 : 1) * p.Hkv) * pairs;
  int64_t group = unroll(bytes, slots, whole_lines(p.D, size)) * kThreads / per_token;
  group = group > p.T / kFewest ? p.T / kFewest : group;
  const int64_t least = (p.T + kMostGroups - 1) / kMostGroups;  // 1, or what a dispatch leaves of very many
  group = group < least ? least : group;
  group = group > kMostTokens ? kMostTokens : group;
  group = group > kTableFloats / half ? kTableFloats / half : group;
  p.group = (int32_t)group;
  p.by_pairs = make_div31(pairs);
  p.by_token = make_div31(per_token);
  p.by_half = make_div31(half);
  return bytes;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int32_t rope_qk_apply_axes(const void* q, void* q_out, const void* k, void* k_out, int64_t T, int32_t Hq,
                           int32_t Hkv, int32_t D, int64_t q_stride, int64_t q_out_stride,
                           int64_t k_stride, int64_t k_out_stride, const int32_t* position_ids,
                           int64_t ids_stride, const int32_t* sections, int32_t axes, int32_t layout,
                           double theta, double pos_scale, int32_t dtype, int32_t direction,
                           void* stream) {
  if (dtype != ROPE_F32 && dtype != ROPE_BF16 && dtype != ROPE_F16) return ROPE_EUNSUPPORTED;
  if (T < 0 || T > INT32_MAX || Hq < 0 || Hq > kMaxHeads || Hkv < 0 || Hkv > kMaxHeads) return ROPE_EINVAL;
  AxesParams p;
  if (!set_frequencies(p, D, sections, axes, layout, theta)) return ROPE_EINVAL;
  p.pos_scale = (float)pos_scale;
  if (!(p.pos_scale >= 1.0f) || p.pos_scale > 3e38f) return ROPE_EINVAL;
  if (direction != 1 && direction != -1) return ROPE_EINVAL;
  p.sign = direction > 0 ? 1.0f : -1.0f;
  const int64_t dense_q = (int64_t)Hq * D, dense_k = (int64_t)Hkv * D;
  if (!stride_of(q_stride, dense_q, &p.q_stride) || !stride_of(q_out_stride, dense_q, &p.q_out_stride) ||
      !stride_of(k_stride, dense_k, &p.k_stride) || !stride_of(k_out_stride, dense_k, &p.k_out_stride))
    return ROPE_EINVAL;
  if (axes > 1 && (ids_stride < T || ids_stride > (int64_t)1 << 40)) return ROPE_EINVAL;
  if (T == 0) return ROPE_OK;
  if (Hq + Hkv == 0 || position_ids == nullptr) return ROPE_EINVAL;
  if (Hq > 0 && (q == nullptr || q_out == nullptr || (q == q_out && p.q_stride != p.q_out_stride)))
    return ROPE_EINVAL;
  if (Hkv > 0 && (k == nullptr || k_out == nullptr || (k == k_out && p.k_stride != p.k_out_stride)))
    return ROPE_EINVAL;
  p.q = q;
  p.q_out = q_out;
  p.k = k;
  p.k_out = k_out;
  p.v = nullptr;
  p.v_out = nullptr;
  p.slots = nullptr;
  p.ids = position_ids;
  p.ids_stride = axes > 1 ? ids_stride : 0;
  p.T = (int32_t)T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.axes = axes;
  const int32_t size = dtype == ROPE_F32 ? 4 : 2;
  const int64_t has_q = Hq > 0, has_k = Hkv > 0;
  const int64_t of[] = {(int64_t)D / 2 * size, has_q * p.q_stride * size, has_q * p.q_out_stride * size,
                        has_k * p.k_stride * size, has_k * p.k_out_stride * size,
                        has_q * (int64_t)(uintptr_t)q, has_q * (int64_t)(uintptr_t)q_out,
                        has_k * (int64_t)(uintptr_t)k, has_k * (int64_t)(uintptr_t)k_out};
  const int32_t bytes = set_geometry(p, size, false, of);
  if ((T + p.group - 1) / p.group > kMostGroups) return ROPE_EINVAL;
  return launch_typed<false>(p, bytes, dtype, static_cast<hipStream_t>(stream));
}

int32_t kv_append_slots(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                        void* v_cache, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                        int64_t q_out_stride, int64_t k_stride, int64_t v_stride, int32_t num_pages,
                        int32_t page_size, int64_t page_stride, int64_t slot_stride,
                        int64_t head_stride, const int64_t* slots, const int32_t* position_ids,
                        int64_t ids_stride, const int32_t* sections, int32_t axes, int32_t layout,
                        double theta, double pos_scale, int32_t dtype, void* stream) {
  if (dtype != ROPE_F32 && dtype != ROPE_BF16 && dtype != ROPE_F16) return ROPE_EUNSUPPORTED;
  if (T < 0 || T > INT32_MAX || Hq < 0 || Hq > kMaxHeads || Hkv < 1 || Hkv > kMaxHeads) return ROPE_EINVAL;
  AxesParams p;
  if (!set_frequencies(p, D, sections, axes, layout, theta)) return ROPE_EINVAL;
  p.pos_scale = (float)pos_scale;
  if (!(p.pos_scale >= 1.0f) || p.pos_scale > 3e38f) return ROPE_EINVAL;
  p.sign = 1.0f;
  const int64_t dense_q = (int64_t)Hq * D, dense_k = (int64_t)Hkv * D, most = (int64_t)1 << 40;
  if (!stride_of(q_stride, dense_q, &p.q_stride) || !stride_of(q_out_stride, dense_q, &p.q_out_stride) ||
      !stride_of(k_stride, dense_k, &p.k_stride) || !stride_of(v_stride, dense_k, &p.v_stride))
    return ROPE_EINVAL;
  if (num_pages < 0 || page_size < 1) return ROPE_EINVAL;
  for (const int64_t x : {page_stride, slot_stride, head_stride})
    if (x < 0 || x > most) return ROPE_EINVAL;
  if (axes > 1 && (ids_stride < T || ids_stride > most)) return ROPE_EINVAL;
  if (T == 0) return ROPE_OK;
  if (slots == nullptr || position_ids == nullptr || k == nullptr || v == nullptr) return ROPE_EINVAL;
  if (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return ROPE_EINVAL;
  if (Hq > 0 && q != nullptr && q_out == nullptr) return ROPE_EINVAL;
  const bool has_q = Hq > 0 && q != nullptr;
  if (has_q && q == q_out && p.q_stride != p.q_out_stride) return ROPE_EINVAL;
  p.q = q;
  p.q_out = q_out;
  p.k = k;
  p.k_out = k_cache;
  p.v = v;
  p.v_out = v_cache;
  p.slots = slots;
  p.ids = position_ids;
  p.k_out_stride = 0;
  p.ids_stride = axes > 1 ? ids_stride : 0;
  p.page_stride = page_stride;
  p.slot_stride = slot_stride;
  p.head_stride = head_stride;
  p.num_slots = (int64_t)num_pages * page_size;
  p.page_size = page_size;
  p.by_page = make_div31(page_size);
  p.T = (int32_t)T;
  p.Hq = has_q ? Hq : 0;
  p.Hkv = Hkv;
  p.D = D;
  p.axes = axes;
  const int32_t size = dtype == ROPE_F32 ? 4 : 2;
  const int64_t of[] = {(int64_t)D / 2 * size, p.k_stride * size, p.v_stride * size,
                        page_stride * size, slot_stride * size, head_stride * size,
                        (int64_t)(uintptr_t)k, (int64_t)(uintptr_t)v, (int64_t)(uintptr_t)k_cache,
                        (int64_t)(uintptr_t)v_cache, has_q ? p.q_stride * size : 0,
                        has_q ? p.q_out_stride * size : 0, has_q ? (int64_t)(uintptr_t)q : 0,
                        has_q ? (int64_t)(uintptr_t)q_out : 0};
  const int32_t bytes = set_geometry(p, size, true, of);
  if ((T + p.group - 1) / p.group > kMostGroups) return ROPE_EINVAL;
  return launch_typed<true>(p, bytes, dtype, static_cast<hipStream_t>(stream));
}

}  // extern "C"
