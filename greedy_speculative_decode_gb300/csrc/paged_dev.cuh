// paged_dev.cuh -- what the paged-cache operators share: the addressing of a
// ragged batch's rows, and the 8-bit cache's numbers.
//
// An 8-bit cache holds e4m3 codes and, for each kv head and block of B = 1 or
// 16 positions, one e8m0 exponent byte b (the value 2^(b - 127)).  A block
// whose largest magnitude is a takes the smallest exponent e >= -100 with
// a <= 448 * 2^e (448 is the largest e4m3 value).  A power of two costs an
// e4m3 block no precision (its relative step does not depend on the scale;
// only the subnormal end moves, by less than one binade against a / 448), makes
// every stored value exact in bf16, and turns the scaling of a score or a
// weight into an addition in the exponent.  A block with an infinity or a NaN
// gets the byte 255 and codes of zero: it reads back as NaN throughout.
#pragma once
#include "paged.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr int kExpMinByte = 27;   // 2^-100, the smallest block exponent
constexpr int kExpNaN = 255;

// Exponent byte of a block from the largest |x| of its bf16 values, given as
// bf16 bits with the sign cleared: x = 2^(E - 127) (1 + M / 128) and
// 448 = 1.75 * 2^8, so the exponent is E - 135, or one more for M > 96.
__device__ __forceinline__ int block_exp_byte(uint32_t a) {
  if (a >= 0x7f80u) return kExpNaN;
  const int b = (int)(a >> 7) - 8 + ((a & 127u) > 96u ? 1 : 0);
  return b < kExpMinByte ? kExpMinByte : b;
}

// 2^(b - 127), NaN for 255.
__device__ __forceinline__ float exp_byte_value(uint32_t b) {
  if (b == kExpNaN) return __uint_as_float(0x7fffffffu);
  return __uint_as_float(b == 0 ? 0x00400000u : b << 23);
}
// 2^(127 - b) for a byte the writer makes (27 .. 247), 0 for 255 (whose codes are zero).
__device__ __forceinline__ float exp_byte_inverse(int b) {
  return b == kExpNaN ? 0.0f : __uint_as_float((uint32_t)(254 - b) << 23);
}

// Two fp32 values as e4m3 codes (round to nearest even; the callers' values
// are at most 448 in magnitude), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The codes in the low / high half of a word as an f16 pair (exact).
__device__ __forceinline__ uint32_t f16x2_of_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Sequence of global row r: the last s with row_start[s] <= r (or r / rows
// for a uniform batch), and its index in that sequence.  False for a row
// behind the last sequence.
__device__ __forceinline__ bool find_row(const RowBatch& b, int r, int& seq, int& i) {
  if (b.row_start == nullptr) {
    seq = r / b.rows_each;
    i = r - seq * b.rows_each;
    return seq < b.n_seq;
  }
  if (r >= __ldg(&b.row_start[b.n_seq]) || r < __ldg(&b.row_start[0])) return false;
  int lo = 0, hi = b.n_seq;  // row_start[lo] <= r < row_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(&b.row_start[mid]) <= r) lo = mid; else hi = mid;
  }
  seq = lo;
  i = r - __ldg(&b.row_start[lo]);
  return true;
}

// Position of a sequence's first row (kept where sums with row counts cannot overflow).
__device__ __forceinline__ int first_of(const RowBatch& b, int seq) {
  return min(max(__ldcg(&b.first[seq]), -(1 << 30)), 1 << 30);
}

// Physical page of position pos (>= 0) of a sequence, or -1 with ST_BAD_PAGE
// raised when the table does not reach it or names no page of the pool.
__device__ __forceinline__ int find_page(const RowBatch& b, int n_pages, int seq, int pos, int* status) {
  const int lp = pos / kPage;
  int page = -1;
  if (lp < b.table_stride && (b.cap == nullptr || pos < __ldcg(b.cap))) page = __ldg(&b.table[(size_t)seq * b.table_stride + lp]);
  if (page < 0 || page >= n_pages) {
    if (status) atomicOr(status, ST_BAD_PAGE);
    return -1;
  }
  return page;
}

}  // namespace
}  // namespace sv
