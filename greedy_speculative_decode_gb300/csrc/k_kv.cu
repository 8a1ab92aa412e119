// k_kv.cu -- rows of K and V into a paged cache and back.
//
// Both directions are bound by memory: per row and kv head they move 2 D
// bf16 values on one side and 2 D codes (and exponents) on the other, with a
// handful of instructions per value.  8 kv heads of 128, 8 bits: 8191 rows
// written in 11.8 us (50 MB moved, 4.3 TB/s), 48 runs of up to 61 rows with an
// exponent a page in 9.5 us, 24 runs of up to 700 fetched in 13.7 us (62 MB,
// 4.5 TB/s); a few rows in 2.6 us, a launch and one wait for memory.
#include "paged.h"
#include "paged_dev.cuh"

#include <cuda_fp16.h>

namespace sv {
namespace {

// |x| of two bf16 pairs, the larger of each half.
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t absmax8(const uint4& x) {
  const uint32_t m = __vmaxu2(absmax2(x.x, x.y), absmax2(x.z, x.w));
  return max(m & 0xffffu, m >> 16);
}

__device__ __forceinline__ float2 floats_of(uint32_t f16x2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
}

// Eight bf16 values times `inv` as e4m3 codes.
__device__ __forceinline__ uint2 codes8(const uint4& x, float inv, bool zero) {
  if (zero) return make_uint2(0u, 0u);
  auto two = [&](uint32_t w) {
    return e4m3x2(__fmul_rn(__uint_as_float(w << 16), inv), __fmul_rn(__uint_as_float(w & 0xffff0000u), inv));
  };
  return make_uint2(two(x.x) | (two(x.y) << 16), two(x.z) | (two(x.w) << 16));
}

template <bool kPaged>
__device__ __forceinline__ const uint4* src_row(const bf16* x, int64_t stride, const KvSource& src, int r, int pos,
                                                int h, int H, int D) {
  if (kPaged)
    return reinterpret_cast<const uint4*>(
        x + (((size_t)(pos / kPage % src.src_pages) * H + h) * kPage + pos % kPage) * D);
  return reinterpret_cast<const uint4*>(x + (int64_t)r * stride + h * D);
}

// Where a row's K and V of one kv head lie: D / 8 lanes move a (row, kv head),
// 16 bytes of bf16 each, and take HB heads of their row at once, so that the row
// is looked up once and 2 HB loads are in flight before the first is used.  (One
// head at a time wrote the 8191 rows in 20.6 us and fetched the 24 runs in 18.4.)
template <int D, int HB>
struct RowUnit {
  static constexpr int L = D / 8;
  int r, h0, lane, pos, page;
  bool inside;  // a row of some sequence
  __device__ __forceinline__ RowUnit(const KvPool& c, const RowBatch& b, int* status) {
    const uint32_t u = blockIdx.x * (256 / L) + threadIdx.x / L, per = c.n_kv_heads / HB;
    lane = threadIdx.x % L;
    r = (int)(u / per);
    h0 = (int)(u % per) * HB;
    int seq, i;
    inside = u < (uint32_t)b.n_rows * per && find_row(b, r, seq, i);
    pos = inside ? first_of(b, seq) + i : -1;
    page = pos < 0 ? -1 : find_page(b, c.n_pages, seq, pos, lane == 0 ? status : nullptr);
  }
  // the pool's row of head h0 + x
  __device__ __forceinline__ size_t row(const KvPool& c, int x) const {
    return ((size_t)page * c.n_kv_heads + h0 + x) * kPage + pos % kPage;
  }
};

// One exponent for each position (or none: bf16).
template <int D, int FMT, bool kPaged, int HB>
__global__ void __launch_bounds__(256) k_kv_write(const KvPool c, const RowBatch b, const KvSource src, int* status) {
  constexpr int L = D / 8;
  pdl_trigger();
  pdl_wait();
  const RowUnit<D, HB> u(c, b, status);
  uint4 kx[HB], vx[HB];
#pragma unroll
  for (int x = 0; x < HB; ++x) {
    kx[x] = vx[x] = make_uint4(0u, 0u, 0u, 0u);
    if (u.page < 0) continue;
    kx[x] = __ldcg(src_row<kPaged>(src.k, src.k_stride, src, u.r, u.pos, u.h0 + x, c.n_kv_heads, D) + u.lane);
    vx[x] = __ldcg(src_row<kPaged>(src.v, src.v_stride, src, u.r, u.pos, u.h0 + x, c.n_kv_heads, D) + u.lane);
  }
#pragma unroll
  for (int x = 0; x < HB; ++x) {
    if (FMT == SV_KV_BF16) {
      if (u.page < 0) continue;
      reinterpret_cast<uint4*>(c.k)[u.row(c, x) * L + u.lane] = kx[x];
      reinterpret_cast<uint4*>(c.v)[u.row(c, x) * L + u.lane] = vx[x];
      continue;
    }
    // both magnitudes in one word, so one reduction serves K and V
    uint32_t m = absmax8(kx[x]) | (absmax8(vx[x]) << 16);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (u.page < 0) continue;
    const int bk = block_exp_byte(m & 0xffffu), bv = block_exp_byte(m >> 16);
    const size_t row = u.row(c, x);
    reinterpret_cast<uint2*>(c.k)[row * L + u.lane] = codes8(kx[x], exp_byte_inverse(bk), bk == kExpNaN);
    reinterpret_cast<uint2*>(c.v)[row * L + u.lane] = codes8(vx[x], exp_byte_inverse(bv), bv == kExpNaN);
    if (u.lane == 0) {
      c.k_exp[row] = (uint8_t)bk;
      c.v_exp[row] = (uint8_t)bv;
    }
  }
}

// One exponent for each page.  A block of 16 x D / 8 threads takes a page of
// one kv head (blockIdx.z: K or V), thread (slot, lane) 8 elements of one
// position.  A page is taken by the first row of the call that lies in it:
// blockIdx.x covers `chunk` consecutive rows, which its first threads look up
// side by side, and takes the pages that begin among them.  Positions that the
// page held before keep their codes unless the new rows raise the exponent;
// then they are rounded anew from their stored values (one more rounding, of
// at most half a step of the new scale).
template <int D, bool kPaged>
__global__ void __launch_bounds__(2 * D) k_kv_write_page(const KvPool c, const RowBatch b, const KvSource src,
                                                         int chunk, int* status) {
  constexpr int L = D / 8, W = 16 * L / 32;
  __shared__ uint32_t s_max[W];
  __shared__ int s_page[kPage], s_pos[kPage], s_n[kPage];  // by row of the chunk; page -1: takes none
  const int H = c.n_kv_heads, h = blockIdx.y, tid = threadIdx.x, slot = tid / L, lane = tid % L;
  const bool is_v = blockIdx.z != 0;
  const bf16* x = is_v ? src.v : src.k;
  const int64_t stride = is_v ? src.v_stride : src.k_stride;
  uint8_t* codes = is_v ? c.v : c.k;
  uint8_t* exps = is_v ? c.v_exp : c.k_exp;
  pdl_trigger();
  pdl_wait();
  const int r0 = blockIdx.x * chunk;
  if (tid < chunk) {
    int seq, i, page = -1, pos = -1, n = 0;
    if (r0 + tid < b.n_rows && find_row(b, r0 + tid, seq, i)) {
      pos = first_of(b, seq) + i;
      // the page's first row in this call: at its first slot, or its sequence's first row
      if (pos >= 0 && (pos % kPage == 0 || i == 0)) {
        n = (b.row_start ? __ldg(&b.row_start[seq + 1]) - __ldg(&b.row_start[seq]) : b.rows_each) - i;
        n = min(min(n, kPage - pos % kPage), b.n_rows - (r0 + tid));
        page = find_page(b, c.n_pages, seq, pos, status);
      }
    }
    s_page[tid] = page;
    s_pos[tid] = pos;
    s_n[tid] = n;
  }
  __syncthreads();
  for (int j = 0; j < chunk; ++j) {
    const int page = s_page[j];
    if (page < 0) continue;
    const int r = r0 + j, pos = s_pos[j], a = pos % kPage, z = a + s_n[j];  // slots a .. z - 1 are written
    const size_t ph = (size_t)page * H + h;
    uint2* dst = reinterpret_cast<uint2*>(codes) + (ph * kPage + slot) * L + lane;
    const bool fresh = slot >= a && slot < z;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint2 old = make_uint2(0u, 0u);
    if (fresh)
      v = __ldcg(src_row<kPaged>(x, stride, src, r + slot - a, pos + slot - a, h, H, D) + lane);
    else if (slot < a)
      old = *dst;
    const int b_old = a > 0 ? exps[ph] : 0;
    uint32_t m = absmax8(v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, s_max[w]);
    const int bn = max(block_exp_byte(m), b_old);
    if (fresh) {
      *dst = codes8(v, exp_byte_inverse(bn), bn == kExpNaN);
    } else if (slot < a && bn != b_old) {
      // the stored codes times 2^(old - new), rounded to codes again
      const float f = bn - b_old > 126 ? 0.0f : __uint_as_float((uint32_t)(127 - (bn - b_old)) << 23);
      auto four = [&](uint32_t w) {
        const float2 p = floats_of(f16x2_of_lo(w)), q = floats_of(f16x2_of_hi(w));
        return e4m3x2(__fmul_rn(p.x, f), __fmul_rn(p.y, f)) | (e4m3x2(__fmul_rn(q.x, f), __fmul_rn(q.y, f)) << 16);
      };
      *dst = bn == kExpNaN ? make_uint2(0u, 0u) : make_uint2(four(old.x), four(old.y));
    }
    __syncthreads();  // every thread has read the old exponent and s_max
    if (tid == 0) exps[ph] = (uint8_t)bn;
  }
}

// The reverse.
template <int D, int FMT, int HB>
__global__ void __launch_bounds__(256) k_kv_fetch(const KvPool c, const RowBatch b, bf16* k, int64_t k_stride,
                                                  bf16* v, int64_t v_stride, int* status) {
  constexpr int L = D / 8;
  const RowUnit<D, HB> u(c, b, status);
  if (!u.inside) return;
  uint4* kd = reinterpret_cast<uint4*>(k + (int64_t)u.r * k_stride + u.h0 * D) + u.lane;
  uint4* vd = reinterpret_cast<uint4*>(v + (int64_t)u.r * v_stride + u.h0 * D) + u.lane;
  if (u.page < 0) {  // padding, or no page (reported)
#pragma unroll
    for (int x = 0; x < HB; ++x) kd[x * L] = vd[x * L] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (FMT == SV_KV_BF16) {
    uint4 kx[HB], vx[HB];
#pragma unroll
    for (int x = 0; x < HB; ++x) {
      kx[x] = __ldcg(reinterpret_cast<const uint4*>(c.k) + u.row(c, x) * L + u.lane);
      vx[x] = __ldcg(reinterpret_cast<const uint4*>(c.v) + u.row(c, x) * L + u.lane);
    }
#pragma unroll
    for (int x = 0; x < HB; ++x) {
      kd[x * L] = kx[x];
      vd[x * L] = vx[x];
    }
    return;
  }
  uint2 kc[HB], vc[HB];
  uint32_t be[HB];
#pragma unroll
  for (int x = 0; x < HB; ++x) {
    const size_t row = u.row(c, x), e = c.block == 1 ? row : row / kPage;
    kc[x] = __ldcg(reinterpret_cast<const uint2*>(c.k) + row * L + u.lane);
    vc[x] = __ldcg(reinterpret_cast<const uint2*>(c.v) + row * L + u.lane);
    be[x] = __ldcg(c.k_exp + e) | (uint32_t)__ldcg(c.v_exp + e) << 8;
  }
#pragma unroll
  for (int x = 0; x < HB; ++x) {
    // four significant bits times a power of two: exact in bf16
    auto eight = [](const uint2& w, float f) {
      const float2 a = floats_of(f16x2_of_lo(w.x)), b = floats_of(f16x2_of_hi(w.x));
      const float2 c = floats_of(f16x2_of_lo(w.y)), d = floats_of(f16x2_of_hi(w.y));
      return make_uint4(pack_bf16x2(__fmul_rn(a.x, f), __fmul_rn(a.y, f)), pack_bf16x2(__fmul_rn(b.x, f), __fmul_rn(b.y, f)),
                        pack_bf16x2(__fmul_rn(c.x, f), __fmul_rn(c.y, f)), pack_bf16x2(__fmul_rn(d.x, f), __fmul_rn(d.y, f)));
    };
    kd[x * L] = eight(kc[x], exp_byte_value(be[x] & 255u));
    vd[x * L] = eight(vc[x], exp_byte_value(be[x] >> 8));
  }
}

template <typename... K, typename... A>
cudaError_t launch(void (*kern)(K...), dim3 grid, int threads, cudaStream_t s, bool pdl, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// (kv heads a group of lanes takes: as many as divide the heads, up to four)
int heads_at_once(int H) { return H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1; }

template <int D, bool kPaged, int HB>
cudaError_t write_rows_t(const KvPool& c, const RowBatch& b, const KvSource& src, int* status, cudaStream_t s, bool pdl) {
  const int64_t threads = (int64_t)b.n_rows * (c.n_kv_heads / HB) * (D / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  return c.fmt == SV_KV_BF16 ? launch(k_kv_write<D, SV_KV_BF16, kPaged, HB>, grid, 256, s, pdl, c, b, src, status)
                             : launch(k_kv_write<D, SV_KV_E4M3, kPaged, HB>, grid, 256, s, pdl, c, b, src, status);
}

template <int D, bool kPaged>
cudaError_t write_t(const KvPool& c, const RowBatch& b, const KvSource& src, int* status, cudaStream_t s, bool pdl) {
  if (c.block == 1) {
    switch (heads_at_once(c.n_kv_heads)) {
      case 4: return write_rows_t<D, kPaged, 4>(c, b, src, status, s, pdl);
      case 2: return write_rows_t<D, kPaged, 2>(c, b, src, status, s, pdl);
      default: return write_rows_t<D, kPaged, 1>(c, b, src, status, s, pdl);
    }
  }
  // rows a block looks through for pages to take: a page's worth, fewer when no sequence has as many
  const int chunk = b.max_rows < kPage ? b.max_rows : kPage;
  const dim3 pages((unsigned)((b.n_rows + chunk - 1) / chunk), c.n_kv_heads, 2);
  return launch(k_kv_write_page<D, kPaged>, pages, 2 * D, s, pdl, c, b, src, chunk, status);
}

template <int D, int HB>
cudaError_t fetch_rows_t(const KvPool& c, const RowBatch& b, bf16* k, int64_t ks, bf16* v, int64_t vs, int* status,
                         cudaStream_t s) {
  const int64_t threads = (int64_t)b.n_rows * (c.n_kv_heads / HB) * (D / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  return c.fmt == SV_KV_BF16
             ? launch(k_kv_fetch<D, SV_KV_BF16, HB>, grid, 256, s, false, c, b, k, ks, v, vs, status)
             : launch(k_kv_fetch<D, SV_KV_E4M3, HB>, grid, 256, s, false, c, b, k, ks, v, vs, status);
}

template <int D>
cudaError_t fetch_t(const KvPool& c, const RowBatch& b, bf16* k, int64_t ks, bf16* v, int64_t vs, int* status,
                    cudaStream_t s) {
  switch (heads_at_once(c.n_kv_heads)) {
    case 4: return fetch_rows_t<D, 4>(c, b, k, ks, v, vs, status, s);
    case 2: return fetch_rows_t<D, 2>(c, b, k, ks, v, vs, status, s);
    default: return fetch_rows_t<D, 1>(c, b, k, ks, v, vs, status, s);
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvPool& c, const RowBatch& b, const KvSource& src, int* status, cudaStream_t s,
                            bool pdl) {
  const bool paged = src.src_pages > 0;
  switch (c.head_dim) {
    case 64: return paged ? write_t<64, true>(c, b, src, status, s, pdl) : write_t<64, false>(c, b, src, status, s, pdl);
    case 128:
      return paged ? write_t<128, true>(c, b, src, status, s, pdl) : write_t<128, false>(c, b, src, status, s, pdl);
    case 256:
      return paged ? write_t<256, true>(c, b, src, status, s, pdl) : write_t<256, false>(c, b, src, status, s, pdl);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_fetch(const KvPool& c, const RowBatch& b, bf16* k, int64_t k_stride, bf16* v, int64_t v_stride,
                            int* status, cudaStream_t s) {
  switch (c.head_dim) {
    case 64: return fetch_t<64>(c, b, k, k_stride, v, v_stride, status, s);
    case 128: return fetch_t<128>(c, b, k, k_stride, v, v_stride, status, s);
    case 256: return fetch_t<256>(c, b, k, k_stride, v, v_stride, status, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sv
