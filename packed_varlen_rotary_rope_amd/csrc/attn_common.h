// attn_common.h -- what the attention kernels share on gfx950: the matrix instruction
// and its register layout, the LDS tiles, the plan's layout and small host helpers.
//
// Matrix products use v_mfma_f32_32x32x16 (bf16 or f16 in, fp32 out). With l the lane
// and h = l / 32, one instruction computes C[m][n] += sum_k A[m][k] B[k][n]:
//   A: lane l holds row m = l % 32,    k = 8h .. 8h + 7
//   B: lane l holds column n = l % 32, k = 8h .. 8h + 7
//   C: lane l holds column n = l % 32, rows m = 8 (i / 4) + 4h + i % 4 for register i.
// The order of k does not matter as long as A and B agree, so eight consecutive C
// registers 8s .. 8s+7 (rows 16s + {4h..4h+3, 8+4h..8+4h+3}) serve as a B operand of the
// next product without moving between lanes: its A operand is read in the same order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/attn.h"

namespace attn {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int N>
struct Constant {
  static constexpr int value = N;
};

// Bits 0 and 1 of x, of all lanes of the workgroup's four waves together. lds: 16 bytes
// that may be overwritten once every wave has come here.
__device__ inline uint32_t any_wave(uint32_t x, uint8_t* lds) {
  const uint32_t mine = (__any(x & 1) ? 1 : 0) | (__any(x & 2) ? 2 : 0);
  uint32_t* flags = reinterpret_cast<uint32_t*>(lds);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) flags[threadIdx.x >> 6] = mine;
  __syncthreads();
  const uint32_t found =
      __builtin_amdgcn_readfirstlane(flags[0] | flags[1] | flags[2] | flags[3]);
  if (found) __syncthreads();  // read by all before it is overwritten
  return found;
}

// How a block of keys (rows) is treated: every pair is seen; some are hidden; some are hidden
// and operands may not be finite.
enum Mode : int { kWhole, kMasked, kCareful };

template <typename T>
struct Vec;
template <>
struct Vec<__bf16> {
  typedef __bf16 x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 x8 __attribute__((ext_vector_type(8)));
  static constexpr uint32_t kExpMask = 0x7f807f80u;  // exponent bits of a pair
  static constexpr uint32_t kExpOne = 0x00800080u;   // lowest exponent bit of each
};
template <>
struct Vec<_Float16> {
  typedef _Float16 x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 x8 __attribute__((ext_vector_type(8)));
  static constexpr uint32_t kExpMask = 0x7c007c00u;
  static constexpr uint32_t kExpOne = 0x04000400u;
};
template <typename T>
using x8 = typename Vec<T>::x8;

__device__ inline f32x16 mfma(x8<__bf16> a, x8<__bf16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16 mfma(x8<_Float16> a, x8<_Float16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Round-to-nearest-even narrowing of a pair, as one 32-bit word.
template <typename T>
__device__ inline uint32_t narrow2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, typename Vec<T>::x2));
}

// Registers 8s .. 8s+7 of a C operand, narrowed: the B operand described above.
template <typename T>
__device__ inline x8<T> narrow8(const f32x16& c, int s) {
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = narrow2<T>(c[8 * s + 2 * j], c[8 * s + 2 * j + 1]);
  return __builtin_bit_cast(x8<T>, w);
}

// The two lanes l and l + 32 hold halves of one column: lo and hi are theirs, in both.
__device__ inline void both_halves(float x, float* lo, float* hi) {
  const uint32_t a = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const uint32_t first = r[0], second = r[1];  // a bit cast of r[1] itself would take r[0]
  *lo = __builtin_bit_cast(float, first);
  *hi = __builtin_bit_cast(float, second);
}
__device__ inline float half_max(float x) {
  float a, b;
  both_halves(x, &a, &b);
  return __builtin_fmaxf(a, b);
}
__device__ inline float half_sum(float x) {
  float a, b;
  both_halves(x, &a, &b);
  return a + b;
}

// ---- LDS tiles ---------------------------------------------------------------------------
// A tile is a number of rows of CPR 16-byte chunks (8 elements). Chunk c of row r lies in
// slot c ^ swizzle(r) of its row. LDS serves 256 bytes (16 slots) a cycle, and neither way of
// reading a tile may ask for one slot twice: row-major reads (16 lanes read one chunk of 16
// rows) find 16 consecutive rows in 16 different slots, and transposed reads
// (ds_read_b64_tr_b16: 32 lanes read 4 rows x 64 bytes) find 4 consecutive rows in 4 different
// groups of 4 slots. Rows of 8 chunks lie two to a 256-byte line. (With both reads on 8 of
// the 16 slots, the dK/dV pass of a packed batch took 446 us and not 402.)
template <int CPR>
__device__ inline uint32_t swizzle(uint32_t r) {
  if constexpr (CPR == 8) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
  return (r & 3) << 2 | (r >> 2 & 3);
}

constexpr int keys_per_block(int db) { return db <= 4 ? 64 : 32; }
constexpr int chunks_per_row(int db) { return db <= 2 ? 8 : db <= 4 ? 16 : 32; }

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// One 16-byte chunk (4-byte word) per lane from global memory into LDS, no registers
// between: lane l's lands at dst + 16 l (4 l), dst the same for the whole wave; lanes that are
// not set in `lanes` write nothing. For whole waves in uniform flow: all lanes are active, and
// are again behind it. In assembly because the compiler otherwise waits for every copy in
// flight before each transposed read of LDS, also of a buffer that no copy writes, and breaks
// the loop up where lanes are left out. m0 holds the LDS address and needs one wait state; it is
// declared, which the compiler heeds and warns of. exec holds what it held before.
// Whoever reads the data waits first (wait_copies).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ inline uint32_t lds_address(const uint8_t* p) {
  return (uint32_t)(uintptr_t)(lds_void*)p;
}
__device__ inline void copy_chunk_to_lds(const void* src, uint32_t dst, uint64_t lanes) {
  asm volatile(
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %2\n\tglobal_load_lds_dwordx4 %0, off\n\t"
      "s_mov_b64 exec, -1"
      :
      : "v"(src), "s"(__builtin_amdgcn_readfirstlane(dst)), "s"(lanes)
      : "memory", "m0");
}
__device__ inline void copy_word_to_lds(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(__builtin_amdgcn_readfirstlane(dst))
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Waits until at most LEFT of this wave's copies (and loads) are in flight, the newest.
template <int LEFT>
__device__ inline void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LEFT) : "memory");
}
// Waits until this wave's copies into LDS have landed but for the newest LEFT, then for the
// other waves of the workgroup (and so for theirs). The barrier is the bare one: a
// workgroup's fence would wait for every copy in flight.
template <int LEFT>
__device__ inline void wait_copies_and_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LEFT) : "memory");
}

// The chunks of a tile, 256 (one workgroup) or 64 (one wave) at a time in the order of LDS:
// of thread t, row (i * COUNT + t) / CPR and this chunk of it.
template <int CPR, int COUNT>
__device__ inline uint32_t row_of(int i, uint32_t t) {
  return (i * COUNT + t) / CPR;
}
template <int CPR, int COUNT>
__device__ inline uint32_t chunk_of(int i, uint32_t t) {
  return ((i * COUNT + t) % CPR) ^ swizzle<CPR>(row_of<CPR, COUNT>(i, t));
}

// Ends a step for the scheduler: nothing moves across. The loops below read LDS a step or two
// ahead of its use and begin a copy or two a step, so that neither is waited for.
__device__ inline void step() { __builtin_amdgcn_sched_barrier(0); }

// Row-major operand: chunk c of row r.
template <typename T, int CPR>
__device__ inline x8<T> read_rows(const uint8_t* tile, uint32_t r, uint32_t c) {
  return *reinterpret_cast<const x8<T>*>(tile + r * (CPR * 16) + ((c ^ swizzle<CPR>(r)) << 4));
}

// Transposed operand A of a product over rows: lane l gets column 32 db + l % 32, rows
// r0 + {4h .. 4h+3, 8 + 4h .. 8 + 4h + 3} (r0 a multiple of 16).
template <typename T, int CPR>
__device__ inline x8<T> read_columns(const uint8_t* tile, uint32_t r0, uint32_t db, uint32_t lane) {
  const uint32_t i = lane & 15;
  const uint32_t c = 4 * db + 2 * (lane >> 4 & 1) + (i >> 1 & 1);
  const uint32_t r = r0 + 4 * (lane >> 5) + (i >> 2);
  const uint8_t* a = tile + r * (CPR * 16) + ((c ^ swizzle<CPR>(r)) << 4) + 8 * (i & 1);
  const uint8_t* b =
      tile + (r + 8) * (CPR * 16) + ((c ^ swizzle<CPR>(r + 8)) << 4) + 8 * (i & 1);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(b));
  const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
  return __builtin_bit_cast(x8<T>, (u32x4){l2[0], l2[1], h2[0], h2[1]});
}

// ---- non-finite values in masked places --------------------------------------------------
// A hidden pair has weight 0, but 0 * inf and 0 * NaN are NaN. The kernels take operands as
// they are, look at the sums in the end, and where one is not finite, walk once more in
// kCareful mode: partly masked blocks are then multiplied with cleaned operands, and the values
// that are not finite are added only where they are seen. (Looking every masked block over
// beforehand cost it two to three times its other vector instructions.)
template <int DB>
__device__ inline bool any_nonfinite(const f32x16 (&o)[DB]) {  // in this lane
  float x = 0.0f;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) x = __builtin_fmaf(o[d][i], 0.0f, x);
  return x != x;
}
template <typename T>
__device__ inline x8<T> cleaned(x8<T> v) {  // non-finite elements as 0
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t bad = ((w[j] & Vec<T>::kExpMask) + Vec<T>::kExpOne) & 0x80008000u;
    // 0x8000 of a half -> 0xffff of that half
    w[j] &= ~((bad >> 15) * 0xffffu);
  }
  return __builtin_bit_cast(x8<T>, w);
}

// ---- division by a launch constant -------------------------------------------------------
// floor(n / d) for 0 <= n < 2^31 and 1 <= d < 2^31 as one 64-bit product and a shift (the
// round-up method of Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994): with l = ceil(log2 d), s = 31 + l, m = ceil(2^s / d), the
// excess n (m d - 2^s) / (d 2^s) stays below 1/d; m < 2^32 because d > 2^(l-1).
struct Div31 {
  uint32_t mul, shift;
};
inline Div31 make_div31(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  const uint32_t s = 31 + l;
  return Div31{(uint32_t)((((uint64_t)1 << s) + d - 1) / d), s};
}
__host__ __device__ inline uint32_t div31(uint32_t n, Div31 f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// ---- limits and helpers of the host side --------------------------------------------------
constexpr int32_t kRowTile = ATTN_ROW_TILE;  // packed query rows of a tile
constexpr int32_t kKeyTile = ATTN_KEY_TILE;  // keys of a tile of the dK/dV pass
constexpr int32_t kHeader = ATTN_PLAN_HEADER;
constexpr int32_t kMaxHeads = 4096;
constexpr int32_t kMaxD = 256;
constexpr int64_t kMaxStride = (int64_t)1 << 24;  // elements; 64 rows stay within 32-bit bytes
constexpr int64_t kMaxBlocks = 0x7fffff;          // workgroups of 256 threads in a dispatch

inline bool valid_head_size(int32_t D) { return D >= 8 && D <= kMaxD && D % 8 == 0; }
inline bool valid_heads(int32_t Hq, int32_t Hkv) {
  return Hkv >= 1 && Hq >= Hkv && Hq <= kMaxHeads && Hq % Hkv == 0;
}
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
inline bool valid_dtype16(int32_t dtype) { return dtype == ROPE_BF16 || dtype == ROPE_F16; }
inline bool data_pointer(const void* p) { return p != nullptr && aligned16(p); }
// A token stride in elements (0: dense) as the kernels take it.
inline bool token_stride(int64_t stride, int32_t heads, int32_t D, int64_t* out) {
  *out = stride == 0 ? (int64_t)heads * D : stride;
  return *out >= (int64_t)heads * D && *out < kMaxStride && *out % 8 == 0;
}
constexpr double kLog2e = 1.4426950408889634;
inline bool valid_scale(double s) {  // positive and normal once it is single precision
  const double f = s * kLog2e;
  return f > 1e-37 && f < 3e38;
}
inline int32_t launched() { return hipGetLastError() == hipSuccess ? ROPE_OK : ROPE_ELAUNCH; }

// Whether a plan is of this call's kind and sizes, as its header says: words 0 and 1 count its
// two lists, 2 to 5 are T, G, num_seqs and Hkv, 8 is the kind (6 and 7: attn_plan.hip).
enum PlanKind : int32_t { kPackedPlan = 0x7061636b, kPagedPlan = 0x70616765 };
template <typename P>
__device__ inline bool plan_matches(const P& p, PlanKind kind) {
  return p.plan[2] == p.T && p.plan[3] == p.G && p.plan[4] == p.num_seqs && p.plan[5] == p.Hkv &&
         p.plan[8] == kind;
}

// Bounds of the tiles of a batch, rows of no sequence among them (128 of those a tile).
inline int64_t row_items(int64_t T, int32_t num_seqs, int32_t G) {
  return T * G / kRowTile + 2 * (int64_t)num_seqs + 3;
}
inline int64_t key_items(int64_t T, int32_t num_seqs) {
  return T / kKeyTile + 2 * (int64_t)num_seqs + 3;
}

}  // namespace attn
