// The pages of a cache (fd_paged_attn.h): writing new tokens into them, and their
// bookkeeping - growing, forking, freeing, compacting, copying.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <algorithm>
#include <cstdint>

#include "fd_decode_attn.h"
#include "fd_internal.h"
#include "fd_paged.h"
#include "fd_paged_attn.h"

namespace fd {
namespace {

#include "fd_device.cuh"

// Every kernel here is launched before the one ahead of it on the stream has
// ended (programmatic dependent launch), and waits for that before it touches
// memory: its launch is out of the way by then.
__device__ __forceinline__ void begin_kernel() {
  grid_dependency_wait();
  grid_launch_dependents();
}

// ================================================================== appending

// Tokens of one sequence that fall into one page.
struct Segment {
  int row;      // first row of k_new / v_new
  int n;        // tokens
  int slot;     // first slot that is written
  int page;     // page id; -1: leave the tokens out
};

// Segment number `seg` of sequence b; n = 0 where there is none. The sequence's
// new tokens are rows [r0, r0 + n) at positions [lens[b] - n, lens[b]); with
// `count` the rows behind the first count[b] are left out, and lens[b] counts
// what was granted. Rows outside [0, T) and negative positions are left out.
__device__ __forceinline__ Segment segment_of(const AppendArgs& a, int b, int seg, bool report) {
  Segment s{0, 0, 0, -1};
  long long r0 = b, n = 1;
  if (a.start) {
    r0 = a.start[b];
    n = a.start[b + 1] - r0;
  }
  if (a.count) n = min(n, static_cast<long long>(max(a.count[b], 0)));
  if (n <= 0) return s;
  if (report && seg == 0 && (r0 < 0 || r0 + n > a.T)) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
  const long long at = static_cast<long long>(a.lens[b]) - n;  // position of row r0
  const long long i0 = max(max(0ll, -r0), -at), i1 = min(n, a.T - r0);
  if (i0 >= i1) return s;
  const long long first = at + i0, end = at + i1;
  const long long j = first / a.P + seg;  // column of the table
  const long long p0 = max(first, j * a.P), p1 = min(end, (j + 1) * a.P);
  if (p0 >= p1) return s;
  if (j >= a.max_pages) {
    if (report) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
    return s;
  }
  s.row = static_cast<int>(r0 + (p0 - at));
  s.n = static_cast<int>(p1 - p0);
  s.slot = static_cast<int>(p0 - j * a.P);
  s.page = a.table[static_cast<size_t>(b) * a.max_pages + j];
  if (s.page < 0 || s.page >= a.num_pages) {
    if (report) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
    s.page = -1;
    s.n = 0;
  }
  return s;
}

// Units of work. A sequence that writes n tokens touches at most n / P + 2
// pages, so with first(b) = start[b] / P + 2 b the segments of sequence b have
// the numbers first(b) .. first(b + 1) - 1 to themselves, and a unit finds its
// sequence by a search in `start`.
__device__ __forceinline__ long long first_unit(const AppendArgs& a, int b) {
  return static_cast<long long>(max(a.start[b], 0) / a.P) + 2ll * b;
}

// The last b in [0, B) with first_unit(b) <= unit, found by the whole warp: each
// round tests 32 places at once, so 1024 sequences take two loads.
__device__ __forceinline__ int sequence_of(const AppendArgs& a, long long unit, int lane) {
  int lo = 0, n = a.B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool in = lane * step < n && first_unit(a, b) <= unit;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const int at = m ? 31 - __clz(m) : 0;
    n = min(step, n - at * step);
    lo += at * step;
  }
  return lo;
}

__device__ __forceinline__ Segment find_segment(const AppendArgs& a, long long unit, int lane, bool report) {
  if (!a.start) return segment_of(a, static_cast<int>(unit), 0, report);
  const int b = sequence_of(a, unit, lane);
  const long long seg = unit - first_unit(a, b);
  if (seg < 0 || seg > 0x3fffffff) return Segment{0, 0, 0, -1};
  return segment_of(a, b, static_cast<int>(seg), report);
}

// Least power of two s with amax <= 448 s, at least 2^-126; 0 for amax = 0.
// 448 = 1.75 * 2^8, so s = 2^(e - 8) where amax = m 2^e with m <= 1.75.
__device__ __forceinline__ float block_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

__device__ __forceinline__ uint16_t quantise2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// Codes of 8 values over a power of two (every scale that this writer makes),
// which divides exactly by a product with its reciprocal. All values finite.
__device__ __forceinline__ uint2 quantise8(const uint4& v, float inv) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = quantise2(__uint_as_float(u[i] << 16) * inv, __uint_as_float(u[i] & 0xffff0000u) * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// y is a result rounded to the nearest float, err (its sign, at least) what it
// lacks: the float towards zero of the exact result, with an odd last place if
// that was not exact. E4M3 codes of it are the nearest of the exact result, which
// those of y are not where y was rounded onto the middle of two codes.
__device__ __forceinline__ float sticky(float y, float err) {
  uint32_t u = __float_as_uint(y);
  if (err != 0.f) u = (u - ((__float_as_uint(err) ^ u) >> 31)) | 1u;
  return __uint_as_float(u);
}

// The same for any scale and any values: NaN where x is not finite, 0 where
// s is 0. Out of line: the divisions' code would crowd the rest out of the
// instruction cache.
__device__ __noinline__ uint2 quantise8_any(uint4 v, float s) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    float x[2] = {__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)};
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      if (!isfinite(x[k])) {
        x[k] = __int_as_float(0x7fffffff);
      } else if (s > 0.f) {
        const float y = x[k] / s;
        x[k] = sticky(y, fmaf(-y, s, x[k]));
      } else {
        x[k] = 0.f;
      }
    }
    c[i] = quantise2(x[0], x[1]);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The reciprocal of a power of two in [2^-126, 2^125], else 0.
__device__ __forceinline__ float pow2_reciprocal(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7fffffu) == 0 && u >= 0x00800000u && u < 0x7e800000u ? __uint_as_float(0x7f000000u - u) : 0.f;
}

// The codes of four values, multiplied.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c & 0xffff), __NV_E4M3)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c >> 16), __NV_E4M3)));
  auto by = [&](float x) { return sticky(x * ratio, fmaf(x, ratio, -(x * ratio))); };
  return quantise2(by(a.x), by(a.y)) | (static_cast<uint32_t>(quantise2(by(b.x), by(b.y))) << 16);
}

// The largest of an item's values (WPI warps; all warps of the block call it).
template <int WPI>
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (WPI > 1) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // red may still be read from a call before
    if ((threadIdx.x & 31) == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WPI; ++i) m = max(m, red[warp / WPI * WPI + i]);
  }
  return m;
}

// An item - one head's K or V of a unit - belongs to WPI warps, each thread of
// which holds VPT vectors of 8 elements in registers: the block's largest value
// has to be known before the first code is written, and the tokens are read
// once. A block looks its unit up once for BLOCK / (32 WPI) items.
// Bound by memory: 2 bytes in and 1 out an element.
template <bool KV8, int VPT, int WPI>
__global__ void __launch_bounds__(WPI > 8 ? WPI * 32 : 256, WPI > 16 ? 2 : WPI > 8 ? 3 : 4) append_kernel(const AppendArgs a) {
  constexpr int kBlock = WPI > 8 ? WPI * 32 : 256;
  constexpr int kItems = kBlock / 32 / WPI;
  __shared__ uint32_t red[kBlock / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  begin_kernel();
  const Segment g = find_segment(a, blockIdx.x, lane, blockIdx.y == 0 && tid == 0);
  if (g.n <= 0) return;
  const int t = tid % (32 * WPI);
  const int row_shift = 28 - __clz(a.HS);  // vectors of a row: HS / 8
  for (int item0 = blockIdx.y * kItems; item0 < 2 * a.NKV; item0 += gridDim.y * kItems) {
    const int item = item0 + tid / (32 * WPI);
    const bool there = item < 2 * a.NKV;
    const int w = item & 1, head = item >> 1;
    const int vecs = there ? g.n << row_shift : 0;
    const long long stride = w ? a.stride[1] : a.stride[0];
    const uint16_t* x = (w ? a.x[1] : a.x[0]) + g.row * stride + static_cast<size_t>(head) * a.HS;
    uint4 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = t + i * 32 * WPI, row = at >> row_shift, col = at & ((1 << row_shift) - 1);
      v[i] = make_uint4(0, 0, 0, 0);
      if (at < vecs) v[i] = __ldcs(reinterpret_cast<const uint4*>(x + row * stride + col * 8));
    }
    const size_t block = static_cast<size_t>(g.page) * a.NKV + head;
    const size_t base = (block * a.P + g.slot) * a.HS;
    if constexpr (!KV8) {
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(w ? a.pages[1] : a.pages[0]) + base);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (t + i * 32 * WPI < vecs) to[t + i * 32 * WPI] = v[i];
    } else {
      float* scale = (w ? a.scale[1] : a.scale[0]) + block;
      const float old = there && g.slot > 0 ? *scale : 0.f;
      // the largest |x| by its bits, two at a time
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        m = __vmaxu2(__vmaxu2(__vmaxu2(m, v[i].x & 0x7fff7fffu), __vmaxu2(v[i].y & 0x7fff7fffu, v[i].z & 0x7fff7fffu)),
                     v[i].w & 0x7fff7fffu);
      m = block_max<WPI>(max(m & 0xffffu, m >> 16), red);
      const bool finite = m < 0x7f80u;
      if (!finite) {  // once more, without the values that are not
        m = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t abs2 = u[k] & 0x7fff7fffu;
            m = __vmaxu2(m, abs2 & ~__vcmpgeu2(abs2, 0x7f807f80u));
          }
        }
        m = max(m & 0xffffu, m >> 16);
      }
      // every warp of a block that has several items comes here if one does
      if (WPI == 1 ? !finite : __syncthreads_or(!finite)) m = block_max<WPI>(m, red);
      if (!there) continue;
      const float s = fmaxf(block_scale(__uint_as_float(m << 16)), old);
      uint8_t* pages = static_cast<uint8_t*>(w ? a.pages[1] : a.pages[0]);
      if (g.slot > 0 && s > old) {  // the earlier tokens' codes, rounded to the new scale
        const float ratio = old / s;
        uint4* held = reinterpret_cast<uint4*>(pages + block * a.P * a.HS);
        for (int i = t; i < g.slot * a.HS / 16; i += 32 * WPI) {
          const uint4 c = held[i];
          held[i] = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
        }
      }
      uint2* to = reinterpret_cast<uint2*>(pages + base);
      const float inv = pow2_reciprocal(s);
      if (finite && inv > 0.f) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * 32 * WPI < vecs) to[t + i * 32 * WPI] = quantise8(v[i], inv);
      } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (t + i * 32 * WPI < vecs) to[t + i * 32 * WPI] = quantise8_any(v[i], s);
      }
      if (t == 0) *scale = s;
    }
  }
}

// ================================================================ bookkeeping

// reserve and compact put the pages in order, which takes prefix sums over all
// of refs: one launch of one block, or, above kOneBlockPages pages, of a
// cluster of 8, each block a consecutive range of the pages, the ranges' totals
// exchanged through distributed shared memory (16 sequences, 1100 pages:
// 13.3 us in a cluster that kept its lists in global memory). Measured with the
// free pages at the high end (reserve, 64 sequences) or anywhere (compact), one
// block / cluster: 1000 pages 4.3 / 6.6 and 2.9 / 5.3 us, 4096 pages 6.0 / 6.8
// and 5.1 / 6.3, 8192 pages 7.8 / 6.8 and 7.7 / 6.1, 16384 pages 11.5 / 7.2 and
// 13.6 / 7.2; 131072 pages in a cluster 15.6 and 18.4. A turn of 1024 pages a
// block, its load, scan and two barriers, is what they take.
constexpr int kCluster = 8;
constexpr int kBookThreads = 1024;
constexpr int kOneBlockPages = 6144;
constexpr int kSharedSeqs = 1024;  // sequences whose lists stay in shared memory

__device__ __forceinline__ int page_free(int refs) { return refs <= 0 ? 1 : 0; }

// Exclusive prefix sum over the block; *total gets the sum.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* warp_sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = x;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, i);
    if (lane >= i) inc += y;
  }
  __syncthreads();  // warp_sums may still be read from the scan before
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  static_assert(kBookThreads == 1024, "a lane for each warp's sum");
  T s = warp_sums[lane];
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, i);
    if (lane >= i) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + inc - x;
}

__device__ __forceinline__ int ld_dsmem_int(const int* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return static_cast<int>(v);
}

// This block's range of the pages: consecutive, a multiple of the block's step.
template <int CL>
__device__ __forceinline__ void page_range(int num_pages, int* first, int* last) {
  const long long step = kBookThreads;
  const long long per = ((num_pages + CL - 1ll) / CL + step - 1) / step * step;
  *first = static_cast<int>(min(per * blockIdx.x, static_cast<long long>(num_pages)));
  *last = static_cast<int>(min(per * (blockIdx.x + 1ll), static_cast<long long>(num_pages)));
}

template <int CL>
__device__ __forceinline__ void book_sync() {
  if constexpr (CL > 1) cluster_sync_all();
  else __syncthreads();
}

// Counts the pages of the range for which `want` holds, and gives the number
// of such pages in the ranges before this one and in all of them.
template <int CL, class F>
__device__ __forceinline__ void count_pages(int first, int last, int* mine, int* warp_sums, F want, int* before,
                                            int* all) {
  int n = 0;
#pragma unroll 4
  for (int p = first + static_cast<int>(threadIdx.x); p < last; p += kBookThreads) n += want(p);
  int total;
  block_scan(n, warp_sums, &total);
  if constexpr (CL == 1) {
    *before = 0;
    *all = total;
    return;
  }
  if (threadIdx.x == 0) *mine = total;
  cluster_sync_all();
  int b = 0, t = 0;
  for (int r = 0; r < CL; ++r) {
    const int y = ld_dsmem_int(mine, r);
    if (r < static_cast<int>(blockIdx.x)) b += y;
    t += y;
  }
  *before = b;
  *all = t;
}

// Workspace of reserve, behind the header: four arrays of B ints.
//   begin: free pages handed out to the sequences before (clamped)
//   have:  pages of the row before the call
//   copy:  number of the move, or -1
//   from:  the shared page
// header[0]: pages handed out in all.
template <int CL>
__global__ void __launch_bounds__(kBookThreads)
    reserve_kernel(int* table, int* lens, int* refs, const int* grow, int* granted, int* moves, int* ws, int B,
                   int max_pages, int num_pages, int P) {
  __shared__ int mine, warp_sums[kBookThreads / 32], taken_sh;
  __shared__ long long warp_sums64[kBookThreads / 32];
  __shared__ int lists[4 * kSharedSeqs];
  const int tid = threadIdx.x;
  begin_kernel();
  const bool small = B <= kSharedSeqs;
  int *begin = ws + kPagesHeader, *have = begin + B, *copy = have + B, *from = copy + B;
  if (CL == 1 && small) begin = lists, have = begin + B, copy = have + B, from = copy + B;
  int first, last, before, free_all;
  page_range<CL>(num_pages, &first, &last);
  // what the first chunk of sequences needs is asked for before the pages are counted
  int old0 = 0, grow0 = 0;
  if (blockIdx.x == 0 && tid < B) {
    old0 = lens[tid];
    grow0 = grow ? grow[tid] : 1;
  }
  count_pages<CL>(first, last, &mine, warp_sums, [&](int p) { return page_free(refs[p]); }, &before, &free_all);
  if (blockIdx.x == 0) {
    long long upto = 0;  // pages needed by the sequences before this chunk
    int taken = 0, copies = 0;
    for (int b0 = 0; b0 < B; b0 += kBookThreads) {
      const int b = b0 + tid;
      int old = 0, n = 0, held = 0, src = -1, shared = 0, fits = 1;
      long long need = 0;
      if (b < B) {
        old = max(b0 == 0 ? old0 : lens[b], 0);
        n = max(b0 == 0 ? grow0 : grow ? grow[b] : 1, 0);
        held = old / P + (old % P != 0);
        const long long want = (static_cast<long long>(old) + n + P - 1) / P;
        if (n > 0 && (want > max_pages || held > max_pages)) {
          fits = 0;
        } else if (n > 0 && old % P != 0) {
          src = table[static_cast<size_t>(b) * max_pages + old / P];
          if (src < 0 || src >= num_pages) {
            atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
            fits = 0;
          } else {
            shared = refs[src] > 1;
          }
        }
        if (n > 0 && fits) need = want - held + shared;
      }
      long long chunk;
      const long long at = upto + block_scan(need, warp_sums64, &chunk);
      const bool given = n > 0 && fits && (need == 0 || at + need <= free_all);
      // moves and pages of the granted in one scan: at most 1024 moves and 2^31 pages
      long long both;
      const long long mark = block_scan(given ? (need << 16) + shared : 0ll, warp_sums64, &both);
      const int move = copies + static_cast<int>(mark & 0xffff);
      if (b < B) {
        begin[b] = static_cast<int>(min(at, static_cast<long long>(num_pages)));
        have[b] = held;
        copy[b] = given && shared ? move : -1;
        from[b] = src;
        granted[b] = given ? n : 0;
        if (given) lens[b] = old + n;
        else if (n > 0) atomicOr(&g_device_error, FD_DEVERR_PAGES_EXHAUSTED);
      }
      upto += chunk;
      taken += static_cast<int>(both >> 16);
      copies += static_cast<int>(both & 0xffff);
    }
    if (tid == 0) {
      taken_sh = ws[0] = taken;
      moves[0] = copies;
      moves[1] = free_all - taken;
    }
  }
  book_sync<CL>();
  const int taken = CL == 1 ? taken_sh : __ldcg(ws);
  if (CL > 1 && small) {
    for (int i = tid; i < 4 * B; i += kBookThreads) lists[i] = __ldcg(begin + i);
    begin = lists, have = begin + B, copy = have + B, from = copy + B;
    __syncthreads();
  }
  // the free page of rank r goes to the last sequence with begin <= r
  for (int p0 = first; p0 < last && before < taken; p0 += kBookThreads) {
    const int p = p0 + tid;
    const int is_free = p < last ? page_free(refs[p]) : 0;
    int total;
    const int r = before + block_scan(is_free, warp_sums, &total);
    if (is_free && r < taken) {
      int lo = 0, hi = B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (begin[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int j = r - begin[lo], c = copy[lo], h = have[lo];
      if (c >= 0 && j == 0) {
        table[static_cast<size_t>(lo) * max_pages + h - 1] = p;
        moves[2 + 2 * static_cast<size_t>(c)] = from[lo];
        moves[3 + 2 * static_cast<size_t>(c)] = p;
      } else {
        table[static_cast<size_t>(lo) * max_pages + h + j - (c >= 0)] = p;
      }
      refs[p] = 1;
    }
    before += total;
  }
  book_sync<CL>();  // every block has read refs: now the copied pages lose their rows
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += kBookThreads)
      if (copy[b] >= 0) atomicSub(refs + from[b], 1);
}

// The i-th page in use with a number >= n takes the i-th free number < n, n =
// pages in use. With r = pages in use before page p: a free page p < n is hole
// p - r, and a page in use p >= n is mover r - (pages in use below n).
// ws[r] = p for those movers and ws[p] = r (distinct places, as r < n <= p).
template <int CL>
__global__ void __launch_bounds__(kBookThreads) compact_kernel(int* refs, int* moves, int* ws, int num_pages) {
  __shared__ int mine, holes, warp_sums[kBookThreads / 32];
  const int tid = threadIdx.x;
  begin_kernel();
  int first, last, before, n;
  page_range<CL>(num_pages, &first, &last);
  count_pages<CL>(first, last, &mine, warp_sums, [&](int p) { return 1 - page_free(refs[p]); }, &before, &n);
  int my_holes = 0;
  for (int p0 = first; p0 < last; p0 += kBookThreads) {
    const int p = p0 + tid;
    const int used = p < last ? 1 - page_free(refs[p]) : 0;
    int total;
    const int r = before + block_scan(used, warp_sums, &total);
    if (p < last && !used && p < n) {
      moves[3 + 2 * static_cast<size_t>(p - r)] = p;
      ++my_holes;
    }
    if (used && p >= n) {
      ws[r] = p;
      ws[p] = r;
    }
    before += total;
  }
  int moved;
  block_scan(my_holes, warp_sums, &moved);
  if constexpr (CL > 1) {
    if (tid == 0) holes = moved;
    cluster_sync_all();
    moved = 0;
    for (int r = 0; r < CL; ++r) moved += ld_dsmem_int(&holes, r);
  } else {
    __syncthreads();
  }
  const int below = n - moved;  // pages in use below n
  for (int i = blockIdx.x * kBookThreads + tid; i < moved; i += CL * kBookThreads) {
    const int src = __ldcg(ws + below + i), dst = __ldcg(moves + 3 + 2 * static_cast<size_t>(i));
    moves[2 + 2 * static_cast<size_t>(i)] = src;
    refs[dst] = refs[src];
    refs[src] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    moves[0] = moved;
    moves[1] = num_pages - n;
  }
  if constexpr (CL > 1) cluster_sync_all();  // no block leaves while another reads its shared memory
}

constexpr int kTableThreads = 256;

// Table entries follow the moves of compact_kernel.
__global__ void __launch_bounds__(kTableThreads)
    renumber_kernel(int* table, const int* moves, const int* ws, long long entries, int num_pages) {
  begin_kernel();
  const int n = num_pages - moves[1], below = n - moves[0];
  for (long long i = blockIdx.x * static_cast<long long>(kTableThreads) + threadIdx.x; i < entries;
       i += static_cast<long long>(gridDim.x) * kTableThreads) {
    const int p = table[i];
    if (p < n) continue;
    if (p >= num_pages) {
      atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
      continue;
    }
    // a page that refs calls free is no mover: its entry, which broke the
    // invariant before the call, keeps its number
    const int k = ws[p] - below;
    if (k >= 0 && k < moves[0] && moves[2 + 2 * static_cast<size_t>(k)] == p)
      table[i] = moves[3 + 2 * static_cast<size_t>(k)];
  }
}

__global__ void __launch_bounds__(kTableThreads)
    fork_kernel(const int* table, const int* lens, const int* parent, int* table_out, int* lens_out, int* refs, int B,
                int B_out, int max_pages, int num_pages) {
  begin_kernel();
  const int i = blockIdx.y;  // a row: old, new or both
  int from = -1;
  if (i < B_out) {
    from = parent[i];
    if (from < -1 || from >= B) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
      from = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) lens_out[i] = from >= 0 ? lens[from] : 0;
  }
  for (int j = blockIdx.x * kTableThreads + threadIdx.x; j < max_pages; j += gridDim.x * kTableThreads) {
    int got = -1;
    if (i < B_out) {
      if (from >= 0) {
        got = table[static_cast<size_t>(from) * max_pages + j];
        if (got < 0) got = -1;
        if (got >= num_pages) {
          atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
          got = -1;
        }
      }
      table_out[static_cast<size_t>(i) * max_pages + j] = got;
    }
    // a row that is its own parent changes no count
    if (from == i) continue;
    if (got >= 0) atomicAdd(refs + got, 1);
    if (i < B) {
      const int was = table[static_cast<size_t>(i) * max_pages + j];
      if (was >= 0 && was < num_pages) atomicSub(refs + was, 1);
    }
  }
}

__global__ void __launch_bounds__(kTableThreads)
    free_kernel(int* table, int* lens, int* refs, const int* keep, int window, int max_pages, int num_pages, int P) {
  begin_kernel();
  const int b = blockIdx.y;
  // every thread of the row takes this minimum, before or after it is stored
  const int len = max(*static_cast<volatile int*>(lens + b), 0);
  const int now = keep ? min(len, max(keep[b], 0)) : len;
  const int last = now / P + (now % P != 0);
  const int first = window > 0 ? max(0, now - window) / P : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) lens[b] = now;
  for (int j = blockIdx.x * kTableThreads + threadIdx.x; j < max_pages; j += gridDim.x * kTableThreads) {
    if (j >= first && j < last) continue;
    int* at = table + static_cast<size_t>(b) * max_pages + j;
    const int p = *at;
    if (p == -1) continue;
    *at = -1;
    if (p >= 0 && p < num_pages) atomicSub(refs + p, 1);
    else atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
  }
}

// ==================================================================== copying

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // 16-byte vectors of a thread in flight
constexpr size_t kCopyPiece = static_cast<size_t>(kCopyThreads) * kCopyVecs * 16;

// Work items: (move, layer, K or V, piece of a page).
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(uint4* k, uint4* v, float* ks, float* vs, const int* moves, int room, int layers, int num_pages,
                int NKV, size_t page_vecs, int pieces) {
  begin_kernel();
  const int n = min(max(moves[0], 0), room);
  const long long items = static_cast<long long>(n) * layers * 2 * pieces;
  auto move_of = [&](long long it) {
    const size_t m = static_cast<size_t>((it / pieces >> 1) / layers);
    return make_int2(moves[2 + 2 * m], moves[3 + 2 * m]);
  };
  // looked up an item ahead: a list entry's latency is as long as a piece's
  int2 next = blockIdx.x < items ? move_of(blockIdx.x) : make_int2(0, 0);
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int src = next.x, dst = next.y;
    if (it + gridDim.x < items) next = move_of(it + gridDim.x);
    const int piece = static_cast<int>(it % pieces);
    const long long rest = it / pieces;
    const int w = static_cast<int>(rest & 1);
    const int layer = static_cast<int>((rest >> 1) % layers);
    if (src < 0 || src >= num_pages || dst < 0 || dst >= num_pages) {
      if (threadIdx.x == 0) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
      continue;
    }
    const size_t base = static_cast<size_t>(layer) * num_pages;
    uint4* x = w ? v : k;
    const uint4* from = x + (base + src) * page_vecs;
    uint4* to = x + (base + dst) * page_vecs;
    const size_t i0 = piece * (kCopyPiece / 16) + threadIdx.x;
    uint4 r[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (i0 + j * kCopyThreads < page_vecs) r[j] = from[i0 + j * kCopyThreads];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (i0 + j * kCopyThreads < page_vecs) to[i0 + j * kCopyThreads] = r[j];
    if (ks && piece == 0) {
      float* s = w ? vs : ks;
      for (int h = threadIdx.x; h < NKV; h += kCopyThreads) s[(base + dst) * NKV + h] = s[(base + src) * NKV + h];
    }
  }
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int block, int cluster, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int row_blocks(int max_pages) { return std::min((max_pages + kTableThreads - 1) / kTableThreads, 64); }

template <bool KV8, int VPT, int WPI>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kBlock = WPI > 8 ? WPI * 32 : 256, kItems = kBlock / 32 / WPI;
  const long long units = a.start ? static_cast<long long>(a.T) / a.P + 2ll * a.B : a.B;
  // One block for a unit's items where there are units enough: looking a unit up
  // costs a warp as much as an item of 16 tokens (8 prompts, 8 heads: two blocks
  // a unit 40.6 us).
  const int rounds = std::min((2 * a.NKV + kItems - 1) / kItems, 65535);  // a grid's y; blocks take several items each
  return launch(append_kernel<KV8, VPT, WPI>, dim3(static_cast<unsigned>(units), units >= 1024 ? 1 : rounds), kBlock, 1,
                stream, a);
}

// Warps of an item: as many as hold a page's tokens of one head in 8 vectors a
// thread (4 where that is less than a warp's 8). Without `start` an item is one token.
template <bool KV8>
cudaError_t launch_append_type(const AppendArgs& a, cudaStream_t stream) {
  if (!a.start) return launch_append<KV8, 2, 1>(a, stream);
  switch (a.P * a.HS / 2048) {
    case 0: return launch_append<KV8, 4, 1>(a, stream);
    case 1: return launch_append<KV8, 8, 1>(a, stream);
    case 2: return launch_append<KV8, 8, 2>(a, stream);
    case 4: return launch_append<KV8, 8, 4>(a, stream);
    case 8: return launch_append<KV8, 8, 8>(a, stream);
    case 16: return launch_append<KV8, 8, 16>(a, stream);
    default: return launch_append<KV8, 8, 32>(a, stream);
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream) {
  return a.kv8 ? launch_append_type<true>(a, stream) : launch_append_type<false>(a, stream);
}

cudaError_t launch_pages_reserve(int* table, int* lens, int* refs, const int* grow, int* granted, int* moves, int* ws,
                                 int B, int max_pages, int num_pages, int P, cudaStream_t stream) {
  const bool one = num_pages <= kOneBlockPages;
  return launch(one ? reserve_kernel<1> : reserve_kernel<kCluster>, dim3(one ? 1 : kCluster), kBookThreads,
                one ? 1 : kCluster, stream, table, lens, refs, grow, granted, moves, ws, B, max_pages, num_pages, P);
}

cudaError_t launch_pages_fork(const int* table, const int* lens, const int* parent, int* table_out, int* lens_out,
                              int* refs, int B, int B_out, int max_pages, int num_pages, cudaStream_t stream) {
  return launch(fork_kernel, dim3(row_blocks(max_pages), std::max(B, B_out)), kTableThreads, 1, stream, table, lens,
                parent, table_out, lens_out, refs, B, B_out, max_pages, num_pages);
}

cudaError_t launch_pages_free(int* table, int* lens, int* refs, const int* keep, int window, int B, int max_pages,
                              int num_pages, int P, cudaStream_t stream) {
  return launch(free_kernel, dim3(row_blocks(max_pages), B), kTableThreads, 1, stream, table, lens, refs, keep, window,
                max_pages, num_pages, P);
}

cudaError_t launch_pages_compact(int* table, int* refs, int* moves, int* ws, int B, int max_pages, int num_pages,
                                 int sms, cudaStream_t stream) {
  const bool one = num_pages <= kOneBlockPages;
  const cudaError_t e = launch(one ? compact_kernel<1> : compact_kernel<kCluster>, dim3(one ? 1 : kCluster), kBookThreads,
                               one ? 1 : kCluster, stream, refs, moves, ws, num_pages);
  const long long entries = static_cast<long long>(B) * max_pages;
  if (e != cudaSuccess || entries == 0) return e;
  const unsigned blocks = static_cast<unsigned>(std::min((entries + kTableThreads - 1) / kTableThreads, sms * 8ll));
  return launch(renumber_kernel, dim3(blocks), kTableThreads, 1, stream, table, moves, ws, entries, num_pages);
}

cudaError_t launch_pages_copy(void* k, void* v, float* ks, float* vs, const int* moves, int room, int layers,
                              int num_pages, int NKV, size_t page_bytes, int sms, cudaStream_t stream) {
  const int pieces = static_cast<int>((page_bytes + kCopyPiece - 1) / kCopyPiece);
  const long long items = static_cast<long long>(room) * layers * 2 * pieces;
  // Two waves of the eight blocks that an SM holds: blocks do not all copy at one rate, and the second
  // wave goes to the SMs that are ahead. On 152 SMs, free, compact and copy of 230 MB with 8 / 16 / 24 / 32 / 64
  // blocks an SM: 87.6 / 83.6 / 82.7 / 81.7 / 81.2 us; a beam step, whose list is nearly empty, with as
  // many blocks to start for nothing: 10.7 / 11.1 / 12.3 / 13.5 / 15.3 us.
  const unsigned blocks = static_cast<unsigned>(std::min(items, sms * 16ll));
  return launch(copy_kernel, dim3(blocks), kCopyThreads, 1, stream, static_cast<uint4*>(k), static_cast<uint4*>(v), ks,
                vs, moves, room, layers, num_pages, NKV, page_bytes / 16, pieces);
}

cudaError_t read_and_clear_device_error_pages(unsigned int* err) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
  *err |= v;
  return e;
}

}  // namespace fd
