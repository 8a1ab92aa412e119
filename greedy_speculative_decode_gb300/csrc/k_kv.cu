// k_kv.cu -- rows of K and V into a paged cache and back.
//
// Both directions are bound by memory: per row and kv head they move 2 D
// bf16 values on one side and 2 D codes (and exponents) on the other, with a
// handful of instructions per value.
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

// One exponent for each position (or none: bf16).  D / 8 lanes take one
// (row, kv head), 16 bytes of K and of V each: both loads are in flight
// before either is used, and the largest magnitude is a shuffle reduction.
template <int D, int FMT, bool kPaged>
__global__ void __launch_bounds__(256) k_kv_write(const KvPool c, const RowBatch b, const KvSource src, int* status) {
  constexpr int L = D / 8;
  const int H = c.n_kv_heads;
  const uint32_t u = blockIdx.x * (256 / L) + threadIdx.x / L;  // (row, kv head)
  const int lane = threadIdx.x % L;
  pdl_trigger();
  pdl_wait();
  const int r = (int)(u / (uint32_t)H), h = (int)(u % (uint32_t)H);
  int seq = 0, i = 0, page = -1, pos = -1;
  if (u < (uint32_t)b.n_rows * H && find_row(b, r, seq, i)) pos = first_of(b, seq) + i;
  uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
  if (pos >= 0) {
    kx = __ldcg(src_row<kPaged>(src.k, src.k_stride, src, r, pos, h, H, D) + lane);
    vx = __ldcg(src_row<kPaged>(src.v, src.v_stride, src, r, pos, h, H, D) + lane);
    page = find_page(b, c.n_pages, seq, pos, status);
  }
  const size_t row = ((size_t)(page < 0 ? 0 : page) * H + h) * kPage + (pos < 0 ? 0 : pos % kPage);
  if (FMT == SV_KV_BF16) {
    if (page < 0) return;
    reinterpret_cast<uint4*>(c.k)[row * L + lane] = kx;
    reinterpret_cast<uint4*>(c.v)[row * L + lane] = vx;
  } else {
    // both magnitudes in one word, so one reduction serves K and V
    uint32_t m = absmax8(kx) | (absmax8(vx) << 16);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (page < 0) return;
    const int bk = block_exp_byte(m & 0xffffu), bv = block_exp_byte(m >> 16);
    reinterpret_cast<uint2*>(c.k)[row * L + lane] = codes8(kx, exp_byte_inverse(bk), bk == kExpNaN);
    reinterpret_cast<uint2*>(c.v)[row * L + lane] = codes8(vx, exp_byte_inverse(bv), bv == kExpNaN);
    if (lane == 0) {
      c.k_exp[row] = (uint8_t)bk;
      c.v_exp[row] = (uint8_t)bv;
    }
  }
  asm volatile("fence.proxy.async.global;" ::: "memory");  // attention reads the pages through TMA
}

// One exponent for each page.  A block of 16 x D / 8 threads takes a page of
// one kv head (blockIdx.z: K or V), thread (slot, lane) 8 elements of one
// position.  A page is taken by the first row of the call that lies in it:
// blockIdx.x covers `chunk` consecutive rows and takes the pages that begin
// among them.  Positions that the page held before keep their codes unless
// the new rows raise the exponent; then they are rounded anew from their
// stored values (one more rounding, of at most half a step of the new scale).
template <int D, bool kPaged>
__global__ void __launch_bounds__(2 * D) k_kv_write_page(const KvPool c, const RowBatch b, const KvSource src,
                                                         int chunk, int* status) {
  constexpr int L = D / 8, W = 16 * L / 32;
  __shared__ uint32_t s_max[W];
  const int H = c.n_kv_heads, h = blockIdx.y, tid = threadIdx.x, slot = tid / L, lane = tid % L;
  const bool is_v = blockIdx.z != 0;
  const bf16* x = is_v ? src.v : src.k;
  const int64_t stride = is_v ? src.v_stride : src.k_stride;
  uint8_t* codes = is_v ? c.v : c.k;
  uint8_t* exps = is_v ? c.v_exp : c.k_exp;
  pdl_trigger();
  pdl_wait();
  for (int j = 0; j < chunk; ++j) {
    const int r = blockIdx.x * chunk + j;
    int seq, i;
    if (r >= b.n_rows) return;
    if (!find_row(b, r, seq, i)) continue;
    const int pos = first_of(b, seq) + i;
    // the page's first row in this call: at its first slot, or the first row
    // at a position >= 0 of its sequence
    if (pos < 0 || !(pos % kPage == 0 || i == 0)) continue;
    const int n = b.row_start ? __ldg(&b.row_start[seq + 1]) - __ldg(&b.row_start[seq]) : b.rows_each;
    const int a = pos % kPage, z = min(kPage, a + n - i);  // slots a .. z - 1 are written
    const int page = find_page(b, c.n_pages, seq, pos, tid == 0 ? status : nullptr);
    if (page < 0) continue;
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
        const uint32_t lo = f16x2_of_lo(w), hi = f16x2_of_hi(w);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        return e4m3x2(__fmul_rn(p.x, f), __fmul_rn(p.y, f)) | (e4m3x2(__fmul_rn(q.x, f), __fmul_rn(q.y, f)) << 16);
      };
      *dst = bn == kExpNaN ? make_uint2(0u, 0u) : make_uint2(four(old.x), four(old.y));
    }
    __syncthreads();  // every thread has read the old exponent and s_max
    if (tid == 0) exps[ph] = (uint8_t)bn;
    asm volatile("fence.proxy.async.global;" ::: "memory");  // attention reads the pages through TMA
  }
}

// The reverse: D / 8 lanes take one (row, kv head).
template <int D, int FMT>
__global__ void __launch_bounds__(256) k_kv_fetch(const KvPool c, const RowBatch b, bf16* k, int64_t k_stride,
                                                  bf16* v, int64_t v_stride, int* status) {
  constexpr int L = D / 8;
  const int H = c.n_kv_heads;
  const uint32_t u = blockIdx.x * (256 / L) + threadIdx.x / L;  // (row, kv head)
  const int lane = threadIdx.x % L;
  if (u >= (uint32_t)b.n_rows * H) return;
  const int r = (int)(u / (uint32_t)H), h = (int)(u % (uint32_t)H);
  int seq, i;
  if (!find_row(b, r, seq, i)) return;
  const int pos = first_of(b, seq) + i;
  uint4* kd = reinterpret_cast<uint4*>(k + (int64_t)r * k_stride + h * D) + lane;
  uint4* vd = reinterpret_cast<uint4*>(v + (int64_t)r * v_stride + h * D) + lane;
  const int page = pos < 0 ? -1 : find_page(b, c.n_pages, seq, pos, status);
  if (page < 0) {  // padding, or no page (reported)
    *kd = *vd = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const size_t row = ((size_t)page * H + h) * kPage + pos % kPage;
  if (FMT == SV_KV_BF16) {
    *kd = __ldcg(reinterpret_cast<const uint4*>(c.k) + row * L + lane);
    *vd = __ldcg(reinterpret_cast<const uint4*>(c.v) + row * L + lane);
  } else {
    const uint2 kc = __ldcg(reinterpret_cast<const uint2*>(c.k) + row * L + lane);
    const uint2 vc = __ldcg(reinterpret_cast<const uint2*>(c.v) + row * L + lane);
    const size_t e = c.block == 1 ? row : row / kPage;
    const float ks = exp_byte_value(__ldcg(c.k_exp + e)), vs = exp_byte_value(__ldcg(c.v_exp + e));
    auto four = [](uint32_t w, float f, uint32_t& lo2, uint32_t& hi2) {
      const uint32_t lo = f16x2_of_lo(w), hi = f16x2_of_hi(w);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      // four significant bits times a power of two: exact in bf16
      lo2 = pack_bf16x2(__fmul_rn(p.x, f), __fmul_rn(p.y, f));
      hi2 = pack_bf16x2(__fmul_rn(q.x, f), __fmul_rn(q.y, f));
    };
    uint4 ko, vo;
    four(kc.x, ks, ko.x, ko.y);
    four(kc.y, ks, ko.z, ko.w);
    four(vc.x, vs, vo.x, vo.y);
    four(vc.y, vs, vo.z, vo.w);
    *kd = ko;
    *vd = vo;
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

template <int D, bool kPaged>
cudaError_t write_t(const KvPool& c, const RowBatch& b, const KvSource& src, int* status, cudaStream_t s, bool pdl) {
  const int64_t threads = (int64_t)b.n_rows * c.n_kv_heads * (D / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (c.fmt == SV_KV_BF16) return launch(k_kv_write<D, SV_KV_BF16, kPaged>, grid, 256, s, pdl, c, b, src, status);
  if (c.block == 1) return launch(k_kv_write<D, SV_KV_E4M3, kPaged>, grid, 256, s, pdl, c, b, src, status);
  // rows a block looks through for pages to take: a page's worth, fewer when no sequence has as many
  const int chunk = b.max_rows < kPage ? b.max_rows : kPage;
  const dim3 pages((unsigned)((b.n_rows + chunk - 1) / chunk), c.n_kv_heads, 2);
  return launch(k_kv_write_page<D, kPaged>, pages, 2 * D, s, pdl, c, b, src, chunk, status);
}

template <int D>
cudaError_t fetch_t(const KvPool& c, const RowBatch& b, bf16* k, int64_t ks, bf16* v, int64_t vs, int* status,
                    cudaStream_t s) {
  const int64_t threads = (int64_t)b.n_rows * c.n_kv_heads * (D / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  return c.fmt == SV_KV_BF16
             ? launch(k_kv_fetch<D, SV_KV_BF16>, grid, 256, s, false, c, b, k, ks, v, vs, status)
             : launch(k_kv_fetch<D, SV_KV_E4M3>, grid, 256, s, false, c, b, k, ks, v, vs, status);
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
