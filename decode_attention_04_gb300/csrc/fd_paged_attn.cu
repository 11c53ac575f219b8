// Single-token attention over a KV cache kept in pages (fd_paged_attn.h).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "fd_decode_attn.h"
#include "fd_internal.h"
#include "fd_paged.h"
#include "fd_paged_attn.h"

namespace fd {
namespace {

#include "fd_device.cuh"

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

// Live band [lo, len) of sequence b; repaired lengths are reported once.
__device__ __forceinline__ int paged_band(const PagedArgs& a, int b, bool report, int* lo) {
  int len = a.lens[b];
  unsigned flags = 0;
  if (len < 0) {
    flags |= FD_DEVERR_LEN_NEGATIVE;
    len = 0;
  }
  if (len > a.max_pages * a.P) {
    flags |= FD_DEVERR_LEN_CLAMPED;
    len = a.max_pages * a.P;
  }
  if (report && flags) atomicOr(&g_device_error, flags);
  *lo = a.window > 0 ? max(0, len - a.window) : 0;
  return len;
}

constexpr int kThreads = 128;

// One block per (query head, sequence): 128 positions at a time, one thread a
// position for the scores, one thread HS / 128 dims for the output.
__global__ void __launch_bounds__(kThreads) paged_simple_kernel(const PagedArgs a) {
  __shared__ float sq[512], sp[kThreads], red[4];
  __shared__ int spage[kThreads];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int kvh = h / (a.NH / a.NKV);
  const size_t row = (static_cast<size_t>(b) * a.NH + h) * a.HS;
  for (int d = tid; d < a.HS; d += kThreads) sq[d] = bf16_bits_to_f32(a.q[row + d]);
  int lo;
  const int len = paged_band(a, b, h == 0 && tid == 0, &lo);
  float m = kNegInf, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p0 = lo; p0 < len; p0 += kThreads) {
    __syncthreads();
    const int pos = p0 + tid;
    float s = kNegInf;
    int page = -1;
    if (pos < len) {
      page = a.table[static_cast<size_t>(b) * a.max_pages + pos / a.P];
      if (page < 0 || page >= a.num_pages) {
        atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
        page = -1;
      }
    }
    if (page >= 0) {
      const size_t at = ((static_cast<size_t>(page) * a.NKV + kvh) * a.P + pos % a.P) * a.HS;
      float dot = 0.f;
      if (a.kv8) {
        const uint8_t* k = static_cast<const uint8_t*>(a.k) + at;
        for (int d = 0; d < a.HS; ++d) dot += sq[d] * e4m3_to_f32(k[d]);
        dot *= a.k_scale[static_cast<size_t>(page) * a.NKV + kvh];
      } else {
        const uint16_t* k = static_cast<const uint16_t*>(a.k) + at;
        for (int d = 0; d < a.HS; ++d) dot += sq[d] * bf16_bits_to_f32(k[d]);
      }
      s = dot * a.scale_log2;
    }
    float mx = s;
    for (int i = 16; i; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    spage[tid] = page;
    __syncthreads();
    mx = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mx == kNegInf ? 0.f : mx;
    const float alpha = exp2f(m - ref);
    m = mx;
    sp[tid] = page >= 0 ? exp2f(s - ref) : 0.f;
    __syncthreads();
    l *= alpha;
    for (int j = 0; j < 4; ++j) o[j] *= alpha;
    for (int t = 0; t < min(kThreads, len - p0); ++t) {
      if (spage[t] < 0) continue;
      const float p = sp[t];
      l += p;
      const size_t at = ((static_cast<size_t>(spage[t]) * a.NKV + kvh) * a.P + (p0 + t) % a.P) * a.HS;
      const float vs = a.kv8 ? a.v_scale[static_cast<size_t>(spage[t]) * a.NKV + kvh] : 1.f;
      for (int j = 0; j < 4; ++j) {
        const int d = tid + j * kThreads;
        if (d < a.HS)
          o[j] += p * (a.kv8 ? e4m3_to_f32(static_cast<const uint8_t*>(a.v)[at + d]) * vs
                             : bf16_bits_to_f32(static_cast<const uint16_t*>(a.v)[at + d]));
      }
    }
  }
  for (int j = 0; j < 4; ++j) {
    const int d = tid + j * kThreads;
    if (d >= a.HS) continue;
    const float x = l == 0.f ? 0.f : o[j] / l;
    a.out[row + d] = f32_to_bf16_bits(x);
    if (a.out_f32) a.out_f32[row + d] = x;
  }
}

}  // namespace

cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream) {
  paged_simple_kernel<<<dim3(a.NH, a.B), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t set_wait_limit_paged(unsigned long long ns) {
  const unsigned long long v = ns ? ns : 1000000000ull;
  return cudaMemcpyToSymbol(g_wait_limit_ns, &v, sizeof v);
}

cudaError_t read_and_clear_device_error_paged(unsigned int* err) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
  *err |= v;
  return e;
}

}  // namespace fd
