// Single-token attention over a KV cache kept in pages (fd_paged_attn.h), on the
// fifth-generation tensor cores: softmax((q K^T) scale) V with one query token a
// sequence, K and V bf16 or E4M3 with a scale for each page and head.
//
// Work. The live bands of all (sequence, KV head) units lie one behind the
// other in granules of 32 positions; block c of C takes the granules [c, c + 1)
// * ceil(total / C). So every SM reads the same number of bytes whatever the lengths are,
// in one wave, and a block leaves at most two partials: of a band that began
// before its share and of one that goes on behind it. A band inside one share
// is written to the output directly.
//
// A block, per tile of 128 positions (a share's part of one band is a segment):
//   * Warp 0 brings K and V into a ring of shared-memory slots (one slot: the
//     tile's 128 positions x 128 head dims) by TMA, a box of one page's rows
//     (32 at most) and 128 bytes each; lane i looks up and copies box i. The order
//     is K(0), then V(i) and K(i + 1) alternately: the scores of the next tile
//     are computed while the softmax of this one runs.
//   * Warp 1 issues the MMAs from one thread, out of order between the two
//     products, accumulators in tensor memory: S^T (positions x query rows) =
//     K Q^T and O^T (dims x query rows) += V^T P^T. With K as the 128-row
//     operand the tensor cores read every code once, as it lies in the cache: nothing
//     is widened.
//   * Warps 2-5 turn scores into weights, a position a thread.
//
// E4M3 products are exact but for the other operand, which enters as a sum of
// E4M3 terms, each in MMA columns of its own, term i scaled by 16^i so that it
// has E4M3's full range: q = q0 + q1 / 16 (8 significant bits: all that bf16 has),
// w = w0 + w1 / 16 + w2 / 256 (12 bits). The columns are added in fp32 at the end. 48 columns
// instead of 16 cost the tensor cores nothing here: an MMA takes as long as reading its
// 128-row operand. bf16 takes q as it is and w = w0 + w1 (16 bits).
//
// Scales. K's multiplies the score. V's enters the weight, w_p = 2^(t_p - m),
// t_p = s_p log2(e) + log2(vs): m follows the largest t, so that w fits E4M3 whatever
// the scales are, and the row's sum l = sum 2^(s_p log2(e) - m) has the same reference.

#include <cuda.h>  // CUtensorMap (descriptor type only; the encoder comes from the runtime)
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "fd_decode_attn.h"
#include "fd_internal.h"
#include "fd_paged.h"
#include "fd_paged_attn.h"

namespace fd {
namespace {

#include "fd_device.cuh"

// ------------------------------------------------------------- PTX helpers

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (tensor memory) = A * B (+ D when accumulate != 0), one thread issues.
template <bool KV8>
__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                     uint32_t accumulate) {
  if constexpr (KV8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// The mbarrier gets one arrival when every MMA this thread issued so far has
// completed (and stopped reading its shared-memory operands).
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 consecutive 32-bit columns of this warp's 32 tensor-memory lanes; the
// values are there after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// N columns (a multiple of 16), waited for.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_ld16(taddr + i, r + i);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    asm volatile("" : "+r"(r[i]));  // no use before the wait
    v[i] = __uint_as_float(r[i]);
  }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 3-D TMA tile load (x = head dim, y = head and slot of a page, z = page).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Shared-memory matrix descriptor: start address / 16 in bits 0-13, leading
// byte offset / 16 in 16-29, stride byte offset / 16 in 32-45, version 1 in
// 46-47, layout in 61-63 (2: 128-byte swizzle, 4: 64-byte). K-major: the rows of an 8-row
// atom are one swizzle width apart, SBO is the distance between atoms.
// MN-major: LBO is the distance between column blocks of one swizzle width,
// SBO between 8-row groups along K.
template <int SW>
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((8 * SW) >> 4) << 32) | (1ull << 46) | (static_cast<uint64_t>(SW == 128 ? 2 : 4) << 61);
}

// Byte offset of 16-byte piece `piece` of row `row` in rows of SW bytes.
template <int SW>
__device__ __forceinline__ uint32_t swizzled(int row, int piece) {
  return row * SW + ((SW == 128 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3)) << 4);
}

// A named barrier that tells every thread whether `p` held for any.
__device__ __forceinline__ bool named_bar_or(int id, int nthreads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.or.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------- the division of work

constexpr int kGranule = 32;    // positions
constexpr int kLenCache = 1024; // lengths kept in shared memory when there are no more sequences

struct Band {
  int len, lo, granules;  // live positions [lo, len), counted in granules from floor(lo / 32)
};

__device__ __forceinline__ int clamp_len(const PagedArgs& a, int len) {
  return min(max(len, 0), a.max_pages * a.P);
}

__device__ __forceinline__ Band band_from(const PagedArgs& a, int len) {
  Band d;
  d.len = len;
  d.lo = a.window > 0 ? max(0, len - a.window) : 0;
  d.granules = len > 0 ? (len - 1) / kGranule - d.lo / kGranule + 1 : 0;
  return d;
}

// A share's part of one unit's band.
struct Tile {
  int b, kvh;
  int pos;         // first position (a multiple of 32)
  int end;         // positions [max(pos, lo), min(pos + 128, end)) are live in the segment
  int lo;
  int seg;         // number of the segment in this block
  bool first, last;    // of the segment
  bool begins, ends;   // the segment holds the band's first / last granule
  bool ok;
};

// Walks a block's tiles in order.
struct Walk {
  long long g, gend, off;  // granules: next one, the share's end, where sequence b's units begin
  int b;
  Band d;
  Tile t;
  int stop;  // end of the segment, positions
};

__device__ __forceinline__ Band band_of_seq(const PagedArgs& a, const int* cache, int b) {
  return band_from(a, a.B <= kLenCache ? cache[b] : clamp_len(a, a.lens[b]));
}

__device__ __forceinline__ void next_tile(const PagedArgs& a, const int* cache, int T, Walk& w) {
  if (w.t.ok && !w.t.last) {
    w.t.pos += T;
    w.t.first = false;
    w.t.last = w.t.pos + T >= w.stop;
    return;
  }
  if (w.g >= w.gend) {
    w.t.ok = false;
    return;
  }
  while (w.g >= w.off + static_cast<long long>(a.NKV) * w.d.granules) {
    w.off += static_cast<long long>(a.NKV) * w.d.granules;
    w.d = band_of_seq(a, cache, ++w.b);
  }
  const long long in = w.g - w.off;
  const int kvh = static_cast<int>(in / w.d.granules);
  const int g0 = static_cast<int>(in - static_cast<long long>(kvh) * w.d.granules);
  const int take = static_cast<int>(min(static_cast<long long>(w.d.granules - g0), w.gend - w.g));
  w.g += take;
  Tile& t = w.t;
  t.seg += 1;
  t.b = w.b;
  t.kvh = kvh;
  t.lo = w.d.lo;
  t.pos = (w.d.lo / kGranule + g0) * kGranule;
  t.begins = g0 == 0;
  t.ends = g0 + take == w.d.granules;
  // the end of the last granule may lie beyond 2^31 - 1: the band's end does not
  t.end = t.ends ? w.d.len : t.pos + take * kGranule;
  w.stop = t.end;
  t.first = true;
  t.last = t.end - t.pos <= T;
  t.ok = true;
}

// --------------------------------------------------------------------- shapes

constexpr int kTile = 128;     // positions per tile: the M of the score MMA
constexpr int kSoftWarps = 4;  // one TMEM lane quarter each
constexpr int W_COPY = 0, W_MMA = 1, W_SOFT0 = 2;
constexpr int kThreads = (W_SOFT0 + kSoftWarps) * 32;
constexpr int kSoft = kSoftWarps * 32;

constexpr int round16(int x) { return (x + 15) / 16 * 16; }
constexpr int pow2_cols(int x) { return x <= 32 ? 32 : x <= 64 ? 64 : x <= 128 ? 128 : x <= 256 ? 256 : 512; }

template <int HS_, bool KV8_, int NQ_>
struct Cfg {
  static constexpr int HS = HS_, NQ = NQ_;
  static constexpr bool KV8 = KV8_;
  static constexpr int EB = KV8 ? 1 : 2;               // bytes of an element
  static constexpr int DB = HS < 128 ? HS : 128;       // dims per slot
  static constexpr int NB = HS / DB;                   // slots per tensor and tile
  static constexpr int SW = DB * EB < 128 ? DB * EB : 128;  // bytes of a swizzled row
  static constexpr int CH = DB * EB / SW;              // chunks (kTile rows of SW bytes) per slot
  static constexpr int CHUNK = kTile * SW;
  static constexpr int SLOT = CH * CHUNK;
  static constexpr int KSTEP = 32 / EB;                // K of one MMA (32 bytes)
  static constexpr int QT = KV8 ? 2 : 1;               // terms of q
  static constexpr int PT = KV8 ? 3 : 2;               // terms of a weight
  static constexpr int NS = round16(QT * NQ);          // columns of S
  static constexpr int NP = round16(PT * NQ);          // columns of O
  static constexpr int COLS = pow2_cols(2 * NS + NB * NP);
  static constexpr int O_COL = 2 * NS;
  static constexpr int Q_BYTES = NB * CH * NS * SW;
  static constexpr int P_BYTES = NP * kTile * EB;
  static constexpr int Q_STRIDE = (Q_BYTES + 1023) / 1024 * 1024;
  static constexpr int RING_ROOM = 227 * 1024 - 2 * Q_STRIDE - 2 * P_BYTES - 3 * NQ * kSoftWarps * 4 - kLenCache * 4 - 2048;
  static constexpr int RING = RING_ROOM / SLOT < 24 ? RING_ROOM / SLOT : 24;  // slots: all the shared memory there is
  static constexpr int OFF_Q = RING * SLOT;
  static constexpr int OFF_P = OFF_Q + 2 * Q_STRIDE;
  static constexpr int OFF_RED = OFF_P + 2 * P_BYTES;  // f32: [2][NQ][4] tile maxima, [NQ][4] sums
  static constexpr int OFF_QMUL = OFF_RED + 3 * NQ * kSoftWarps * 4;  // f32 [2][16]
  static constexpr int OFF_LEN = OFF_QMUL + 2 * 16 * 4;
  static constexpr int OFF_BAR = OFF_LEN + kLenCache * 4;
  // full[RING], empty[RING], s_full[2], s_free[2], p_ready[2], pv_done[2], q_ready[2], o_free, mma_done,
  // v_clean[2][NB]
  static constexpr int NBAR = 2 * RING + 12 + 2 * NB;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tensor memory address; share; edge[2]
  static constexpr int SMEM = OFF_MISC + 64 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(P_BYTES % 1024 == 0 && OFF_P % 1024 == 0, "swizzle atoms are aligned");
  static_assert(OFF_BAR % 8 == 0, "barriers");
  static_assert(RING >= 4, "K and V slots pass each other");
  // Stream position of slot p of tile t's K and V: K(0), then V(i), K(i + 1)
  // alternately, the last tile's V by itself.
  static __device__ __forceinline__ int seq_k(int t, int p) { return t == 0 ? p : NB + 2 * NB * (t - 1) + 2 * p + 1; }
  static __device__ __forceinline__ int seq_v(int t, int p, bool more) { return NB + 2 * NB * t + (more ? 2 * p : p); }
  // Instruction descriptor: D f32; A and B E4M3 (0) or bf16 (1 in bits 7 and
  // 10); bit 15: A is MN-major; N / 8 at 17, M / 16 at 24.
  static constexpr uint32_t IDESC_QK = (1u << 4) | (KV8 ? 0u : (1u << 7) | (1u << 10)) |
                                       (static_cast<uint32_t>(NS >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
  static constexpr uint32_t IDESC_PV = (1u << 4) | (KV8 ? 0u : (1u << 7) | (1u << 10)) | (1u << 15) |
                                       (static_cast<uint32_t>(NP >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
};

struct MaxOp {
  __device__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
struct AddOp {
  __device__ float operator()(float x, float y) const { return x + y; }
};

// Reduction of N per-thread values (one per query row) over the 32 lanes of a
// warp by halving: each exchange hands half of the rows still held to the
// partner lane. Lane l ends with row l / (32 / N).
template <int N, class Op>
__device__ __forceinline__ float rowreduce(const float (&v)[N], int lane, Op op) {
  float a[N];
#pragma unroll
  for (int j = 0; j < N; ++j) a[j] = v[j];
  int dist = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2) {
    const bool up = lane & dist;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float keep = up ? a[j + n] : a[j], give = up ? a[j] : a[j + n];
      a[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, dist));
    }
    dist >>= 1;
  }
  float r = a[0];
#pragma unroll
  for (int i = 16 / N; i >= 1; i /= 2) r = op(r, __shfl_xor_sync(0xffffffffu, r, i));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
  return __half22float2(__half2(h));
}

// x = c0 + c1 / 16 + c2 / 256 + ...: the next E4M3 term of a pair; x becomes
// what is left, times 16. x is at most 448 in size.
__device__ __forceinline__ uint16_t next_term(float2& x) {
  const uint16_t c = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
  const float2 y = e4m3x2_to_f32(c);
  x.x = (x.x - y.x) * 16.f;
  x.y = (x.y - y.y) * 16.f;
  return c;
}

struct Maps {
  CUtensorMap k, v;
};

// Which units a block's share breaks: written for the merge.
struct Cut {
  int b, kvh;
  int c0, c1;  // the unit lies in the shares c0 .. c1; c0 < 0: the share ends where a unit does
};

// The smallest power of the running reference that is moved: weights are at
// most 2^kLazy times the bias, which keeps them within E4M3's 448.
constexpr float kLazy8 = 4.f, kBias8 = 4.f;
constexpr float kLazy16 = 8.f, kBias16 = 0.f;

template <class C>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ Maps maps, const PagedArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  const int c = blockIdx.x;
  const int G = a.NH / a.NKV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const uint32_t bar0 = base + C::OFF_BAR;
  const uint32_t full = bar0, empty = full + 8 * C::RING;
  const uint32_t s_full = empty + 8 * C::RING, s_free = s_full + 16, p_ready = s_free + 16, pv_done = p_ready + 16;
  const uint32_t q_ready = pv_done + 16, o_free = q_ready + 16, mma_done = o_free + 8, v_clean = mma_done + 8;
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* qmul = reinterpret_cast<float*>(smem + C::OFF_QMUL);
  int* lens = reinterpret_cast<int*>(smem + C::OFF_LEN);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  long long* share = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);  // per, off of b0, total
  int* share_b = reinterpret_cast<int*>(smem + C::OFF_MISC + 40);
  volatile int* edge = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 48);  // of tile i: V has rows to clear

  // Set-up that reads no input, overlapping the previous kernel's tail.
  if (tid == 0) {
    for (int k = 0; k < C::RING; ++k) {
      mbar_init(full + 8 * k, 1);
      mbar_init(empty + 8 * k, 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(s_full + 8 * j, 1);
      mbar_init(s_free + 8 * j, kSoft);
      mbar_init(p_ready + 8 * j, kSoft);
      mbar_init(pv_done + 8 * j, 1);
      mbar_init(q_ready + 8 * j, kSoft);
    }
    mbar_init(o_free, kSoft);
    for (int j = 0; j < 2 * C::NB; ++j) mbar_init(v_clean + 8 * j, kSoft);
    mbar_init(mma_done, 1);
    fence_mbar_init();
    prefetch_tensor_map(&maps.k);
    prefetch_tensor_map(&maps.v);
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // The total of granules, then the sequence in which this block's share begins.
  {
    long long* sums = reinterpret_cast<long long*>(smem + C::OFF_RED);  // [kThreads / 32]
    long long mine = 0;
    unsigned flags = 0;
    for (int b = tid; b < a.B; b += kThreads) {
      const int raw_len = a.lens[b], len = clamp_len(a, raw_len);
      if (raw_len < 0) flags |= FD_DEVERR_LEN_NEGATIVE;
      if (raw_len > len) flags |= FD_DEVERR_LEN_CLAMPED;
      if (a.B <= kLenCache) lens[b] = len;
      mine += band_from(a, len).granules;
    }
    if (c == 0 && flags) atomicOr(&g_device_error, flags);
    long long s = mine;
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < kThreads / 32; ++i) total += sums[i];
    total *= a.NKV;
    const long long per = max((total + a.blocks - 1) / a.blocks, static_cast<long long>(a.min_share));
    const long long start = per * c;
    if (tid == 0) {
      share[0] = per;
      share[2] = total;
    }
    long long before = 0;  // granules (of one head) of the sequences before this chunk
    for (int b0 = 0; b0 < a.B && start < total; b0 += kThreads) {
      const int b = b0 + tid;
      const long long x = b < a.B ? band_of_seq(a, lens, b).granules : 0;
      long long inc = x;
      for (int i = 1; i < 32; i <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, i);
        if (lane >= i) inc += y;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      long long all = 0;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) inc += sums[i];
        all += sums[i];
      }
      const long long off = (before + inc - x) * a.NKV;
      if (x > 0 && off <= start && start < off + x * a.NKV) {
        share[1] = off;
        *share_b = b;
      }
      before += all;
      if (start < before * a.NKV) break;
    }
    __syncthreads();
  }
  const long long per = share[0], total = share[2];
  Walk walk;
  walk.g = min(per * c, total);
  walk.gend = min(per * (c + 1), total);
  walk.t.ok = false;
  walk.t.seg = -1;
  const bool work = walk.g < walk.gend;
  if (work) {
    walk.off = share[1];
    walk.b = *share_b;
    walk.d = band_of_seq(a, lens, walk.b);
    next_tile(a, lens, kTile, walk);
  }

  // Rows of empty sequences are zero.
  for (int b = c; b < a.B; b += gridDim.x) {
    if ((a.B <= kLenCache ? lens[b] : clamp_len(a, a.lens[b])) > 0) continue;
    for (int i = tid; i < a.NH * C::HS; i += kThreads) {
      const size_t o = static_cast<size_t>(b) * a.NH * C::HS + i;
      a.out[o] = 0;
      if (a.out_f32) a.out_f32[o] = 0.f;
    }
  }
  Cut* cuts = reinterpret_cast<Cut*>(a.cuts);
  if (!work) {
    if (tid == 0) cuts[c].c0 = -1;
    return;
  }

  bool failed = false;
  uint32_t tmem = 0;
  if (warp >= W_MMA) {
    if (warp == W_MMA) {
      tmem_alloc(base + C::OFF_MISC, C::COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(2, (1 + kSoftWarps) * 32);
    tc_fence_after();
    tmem = *tmem_at;
  }

  if (warp == W_COPY) {
    // ------------------------------------------------------------ copy warp
    const int box = min(a.P, 32);           // rows of a copy
    const int nbox = kTile / box;
    const uint32_t box_bytes = box * C::SW * C::CH;
    // the table's entry for this lane's box in a tile; -1: nothing to copy
    auto page_of = [&](const Tile& t) {
      const int r = lane * box;
      if (!t.ok || lane >= nbox || r >= t.end - t.pos || t.pos + r + box <= t.lo) return -1;
      return a.table[static_cast<size_t>(t.b) * a.max_pages + (t.pos + r) / a.P];
    };
    Tile cur = walk.t;
    int cur_page = page_of(cur);
    next_tile(a, lens, kTile, walk);
    Tile nxt = walk.t;
    int nxt_page = page_of(nxt);
    int e = 0, slot = 0, use = 0;
    uint32_t st_issued = 0, st_par = 0;
    auto copy = [&](const Tile& t, int page, bool is_k, int p) {
      if (use > 0) mbar_wait(empty + 8 * slot, (use - 1) & 1, failed);
      const uint32_t fb = full + 8 * slot;
      const bool there = page >= 0 && page < a.num_pages;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, there));
      if (lane == 0) mbar_arrive_expect_tx(fb, boxes * box_bytes);
      __syncwarp();
      if (there) {
        const int r = lane * box;
        const int y = t.kvh * a.P + (t.pos + r) % a.P;
#pragma unroll
        for (int ch = 0; ch < C::CH; ++ch)
          tma_load_3d(base + slot * C::SLOT + ch * C::CHUNK + r * C::SW, is_k ? &maps.k : &maps.v,
                      p * C::DB + ch * (C::SW / C::EB), y, page, fb);
      }
      st_issued |= 1u << slot;
      st_par = (st_par & ~(1u << slot)) | (static_cast<uint32_t>(use & 1) << slot);
      ++e;
      if (++slot == C::RING) {
        slot = 0;
        ++use;
      }
    };
    for (int p = 0; p < C::NB; ++p) copy(cur, cur_page, true, p);
    while (cur.ok) {
      // the pages of the tile after the next are looked up while these copies wait for slots
      next_tile(a, lens, kTile, walk);
      const Tile after = walk.t;
      const int after_page = page_of(after);
      for (int p = 0; p < C::NB; ++p) {
        copy(cur, cur_page, false, p);
        if (nxt.ok) copy(nxt, nxt_page, true, p);
      }
      cur = nxt;
      cur_page = nxt_page;
      nxt = after;
      nxt_page = after_page;
    }
    // No copy may be in flight when the block leaves (bounded, own flag).
    bool dfail = false;
    for (int k = 0; k < C::RING; ++k)
      if ((st_issued >> k) & 1u) mbar_wait(full + 8 * k, (st_par >> k) & 1u, dfail);
  } else if (warp == W_MMA) {
    // ----------------------------------------------------- MMA issue thread
    if (lane == 0) {
      Walk vw = walk;
      int kt = 0, kp = 0, vt = 0, vp = 0;
      bool s_ok = false, p_ok = false, clear = false;
      uint32_t cleared = 0;  // bit j: parity of the phase of tiles of parity j
      uint64_t t_idle = 0;
      uint32_t spins = 0;  // polls without progress; the clock is read every 4096
      while (vw.t.ok && !failed) {
        bool prog = false;
        if (walk.t.ok) {
          // the S buffer is free, and the segment's query rows are in place
          if (!s_ok) s_ok = (kt < 2 || mbar_test(s_free + 8 * (kt & 1), ((kt - 2) >> 1) & 1)) &&
                            (!walk.t.first || mbar_test(q_ready + 8 * (walk.t.seg & 1), (walk.t.seg >> 1) & 1));
          const int e = C::seq_k(kt, kp), slot = e % C::RING;
          if (s_ok && mbar_test(full + 8 * slot, (e / C::RING) & 1)) {
            tc_fence_after();
            const uint32_t kb = base + slot * C::SLOT;
            const uint32_t qb = base + C::OFF_Q + (walk.t.seg & 1) * C::Q_STRIDE + kp * C::CH * C::NS * C::SW;
#pragma unroll
            for (int ch = 0; ch < C::CH; ++ch)
#pragma unroll
              for (int kk = 0; kk < C::SW / 32; ++kk)
                umma<C::KV8>(tmem + C::NS * (kt & 1), smem_desc<C::SW>(kb + ch * C::CHUNK + 32 * kk, 16),
                             smem_desc<C::SW>(qb + ch * C::NS * C::SW + 32 * kk, 16), C::IDESC_QK,
                             (kp | ch | kk) != 0);
            umma_commit(empty + 8 * slot);
            if (++kp == C::NB) {
              umma_commit(s_full + 8 * (kt & 1));
              kp = 0;
              ++kt;
              s_ok = false;
              next_tile(a, lens, kTile, walk);
            }
            prog = true;
          }
        }
        if (vt < kt) {
          // the weights are in place, and the segment before has left O
          if (!p_ok) {
            p_ok = mbar_test(p_ready + 8 * (vt & 1), (vt >> 1) & 1) &&
                   (!vw.t.first || vw.t.seg == 0 || mbar_test(o_free, (vw.t.seg - 1) & 1));
            if (p_ok) clear = edge[vt & 1] != 0;
          }
          const int e = C::seq_v(vt, vp, kt > vt + 1 || walk.t.ok), slot = e % C::RING;
          if (p_ok && mbar_test(full + 8 * slot, (e / C::RING) & 1) && (!clear || mbar_test(v_clean + 8 * ((vt & 1) * C::NB + vp), (cleared >> (vt & 1)) & 1))) {
            tc_fence_after();
            const uint32_t vb = base + slot * C::SLOT;
            const uint32_t pb = base + C::OFF_P + (vt & 1) * C::P_BYTES;
            const uint32_t d = tmem + C::O_COL + C::NP * vp;
            const int nk = (min(kTile, vw.t.end - vw.t.pos) + C::KSTEP - 1) / C::KSTEP;
            for (int kk = 0; kk < nk; ++kk) {
              const uint32_t pa = pb + kk * 32 / 128 * (C::NP * 128) + kk * 32 % 128;
              umma<C::KV8>(d, smem_desc<C::SW>(vb + kk * C::KSTEP * C::SW, C::CH > 1 ? C::CHUNK : C::SLOT),
                           smem_desc<128>(pa, 16), C::IDESC_PV, (!vw.t.first || kk > 0) ? 1u : 0u);
            }
            umma_commit(empty + 8 * slot);
            if (++vp == C::NB) {
              umma_commit(pv_done + 8 * (vt & 1));
              if (clear) cleared ^= 1u << (vt & 1);
              vp = 0;
              ++vt;
              p_ok = false;
              next_tile(a, lens, kTile, vw);
            }
            prog = true;
          }
        }
        if (prog) {
          spins = 0;
        } else if ((++spins & 4095u) == 0) {
          const uint64_t now = globaltimer_ns();
          if (spins == 4096u) {
            t_idle = now;
          } else if (now - t_idle > g_wait_limit_ns) {
            failed = true;
            atomicOr(&g_device_error, FD_DEVERR_WAIT_TIMEOUT);
          }
        }
      }
      // every MMA issued has completed before the tensor memory is released
      umma_commit(mma_done);
      bool dfail = false;
      mbar_wait(mma_done, 0, dfail);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------- softmax / epilogue warps
    constexpr float kLazy = C::KV8 ? kLazy8 : kLazy16, kBias = C::KV8 ? kBias8 : kBias16;
    const int sw = warp - W_SOFT0;
    const int quarter = warp & 3;   // the TMEM lane quarter this warp may access
    const int tq = tid - W_SOFT0 * 32;
    const int pl = quarter * 32 + lane;  // the tile's position whose scores this thread holds
    const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;

    // Query rows of a segment -> the B operand of its score MMAs: rows of SW bytes, swizzled,
    // term j of row r in row j * NQ + r; rows >= G are zero.
    auto stage_q = [&](const Tile& t) {
      const int par = t.seg & 1;
      unsigned char* qb = smem + C::OFF_Q + par * C::Q_STRIDE;
      constexpr int EL = 16 / C::EB;           // elements of a 16-byte piece
      constexpr int PIECES = C::HS / EL;       // of a row: a power of two, at most 64
      for (int id = tq; (id & ~31) < C::NQ * PIECES; id += kSoft) {  // whole warps
        const int r = id / PIECES, pc = id % PIECES;
        const bool live = r < G && r < C::NQ;
        const int chunk = pc * 16 / C::SW, piece = (pc * 16 % C::SW) / 16;
        const uint16_t* src = a.q + (static_cast<size_t>(t.b) * a.NH + static_cast<size_t>(t.kvh) * G + r) * C::HS + pc * EL;
        if constexpr (!C::KV8) {
          if (r < C::NQ)
            *reinterpret_cast<uint4*>(qb + chunk * C::NS * C::SW + swizzled<C::SW>(r, piece)) =
                live ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
        } else {
          uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if (live) {
            x[0] = reinterpret_cast<const uint4*>(src)[0];
            x[1] = reinterpret_cast<const uint4*>(src)[1];
          }
          const uint32_t* u = reinterpret_cast<const uint32_t*>(x);
          float2 f[8];
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
            top = fmaxf(top, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
          }
          // the row's largest element, over the lanes that hold the row
#pragma unroll
          for (int i = PIECES / 2; i >= 1; i /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
          // times a power of two that brings it to [128, 256); not finite: as it is
          const int ex = static_cast<int>(__float_as_uint(top) >> 23);  // biased exponent of top >= 0
          const int sh = (top > 0.f && ex < 255) ? min(7 - (ex - 127), 126) : 0;
          const float mul = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
          if (pc == 0 && r < C::NQ) qmul[par * 16 + r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
          uint32_t w[2][4];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 y = make_float2(f[i].x * mul, f[i].y * mul);
            // an infinity would saturate: it has to reach the scores as NaN
            if (ex == 255) {
              y.x = isfinite(y.x) ? y.x : __int_as_float(0x7fffffff);
              y.y = isfinite(y.y) ? y.y : __int_as_float(0x7fffffff);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t term = next_term(y);
              if (i & 1) w[j][i / 2] |= term << 16;
              else w[j][i / 2] = term;
            }
          }
          if (r < C::NQ) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<uint4*>(qb + chunk * C::NS * C::SW + swizzled<C::SW>(j * C::NQ + r, piece)) =
                  make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(q_ready + 8 * par);
    };

    // Of this thread's position: the table's entry, two tiles ahead, and the
    // block's scales, one tile ahead: both are in flight while a tile is worked on. -1: the position takes no part.
    auto entry = [&](const Tile& t) {
      const int pos = t.pos + pl;
      if (!t.ok || pl >= t.end - t.pos || pos < t.lo) return -1;
      return a.table[static_cast<size_t>(t.b) * a.max_pages + pos / a.P];
    };
    auto scales = [&](const Tile& t, int page) {
      if (!C::KV8 || page < 0 || page >= a.num_pages) return make_float2(0.f, 0.f);
      const size_t at = static_cast<size_t>(page) * a.NKV + t.kvh;
      return make_float2(a.k_scale[at], a.v_scale[at]);
    };

    Tile cur = walk.t;
    int page = entry(cur);
    next_tile(a, lens, kTile, walk);
    Tile nxt = walk.t;
    int next_page = entry(nxt);
    Walk ahead = walk;  // runs to the first tile of the next segment
    stage_q(cur);
    named_bar_sync(1, kSoft);  // qmul
    float2 ksvs = scales(cur, page);
    float m_use[C::NQ], l_part[C::NQ];
    int i = 0;
    while (cur.ok) {
      next_tile(a, lens, kTile, walk);
      const Tile after = walk.t;
      const int after_page = entry(after);
      const float2 next_ksvs = scales(nxt, next_page);
      if (cur.first) {
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) {
          m_use[r] = kNegInf;
          l_part[r] = 0.f;
        }
        // The next segment's query rows; their buffer was last read by the scores of
        // the segment before this one, which have been waited for.
        if (ahead.t.ok && !ahead.t.first) {
          ahead.t.last = true;
          next_tile(a, lens, kTile, ahead);
        }
        if (ahead.t.ok) {
          stage_q(ahead.t);
          next_tile(a, lens, kTile, ahead);
        }
      }
      const bool live = page >= 0 && page < a.num_pages;
      const int rows = (min(kTile, cur.end - cur.pos) + C::KSTEP - 1) / C::KSTEP * C::KSTEP;  // that P.V reads
      const bool dead_row = !live && pl < rows;
      if (dead_row && cur.pos + pl >= cur.lo && cur.pos + pl < cur.end) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
      mbar_wait(s_full + 8 * (i & 1), (i >> 1) & 1, failed);
      tc_fence_after();
      float s[C::NS];
      tmem_load<C::NS>(tmem + tlane + C::NS * (i & 1), s);
      tc_fence_before();
      mbar_arrive(s_free + 8 * (i & 1));

      // sc: log2 of the weight for the row's sum; sc + lvs: for the product with V's codes
      float sc[C::NQ], t[C::NQ];
      float lvs = 0.f;
      if constexpr (C::KV8) {
        // a scale of 0 counts as 2^-150: its weights vanish beside any other's
        lvs = ksvs.y == 0.f ? -150.f : log2f(ksvs.y);
#pragma unroll
        for (int r = 0; r < C::NQ; ++r)
          sc[r] = (s[r] + s[C::NQ + r] * 0.0625f) * (ksvs.x * qmul[(cur.seg & 1) * 16 + r]);
      } else {
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) sc[r] = s[r] * a.scale_log2;
      }
#pragma unroll
      for (int r = 0; r < C::NQ; ++r) {
        sc[r] = live ? sc[r] : kNegInf;
        t[r] = sc[r] + lvs;
      }
      // the tile's row maxima: warp butterfly, then the four warps' values
      float* rm = red + (i & 1) * C::NQ * kSoftWarps;
      const float wmax = rowreduce<C::NQ>(t, lane, MaxOp());
      constexpr int kPer = 32 / C::NQ;  // lanes that end with the same row
      if (lane % kPer == 0) rm[(lane / kPer) * kSoftWarps + sw] = wmax;
      const bool clear = named_bar_or(1, kSoft, dead_row);  // the same for every thread
      bool resc = false;
      float alpha[C::NQ];
#pragma unroll
      for (int r = 0; r < C::NQ; ++r) {
        const float4 t4 = *reinterpret_cast<const float4*>(rm + r * kSoftWarps);
        const float mt = fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
        const bool need = mt > m_use[r] + kLazy;  // false for -inf and NaN
        alpha[r] = need ? exp2f(m_use[r] - mt) : 1.f;
        if (need) m_use[r] = mt;
        resc |= need;
      }
      // every thread took the same decision from the same shared values
      if (resc) {
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) l_part[r] *= alpha[r];
        if (!cur.first) {  // O holds the segment's earlier tiles: rescale it once P.V(i - 1) is done
          mbar_wait(pv_done + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, failed);
          tc_fence_after();
#pragma unroll
          for (int mb = 0; mb < C::NB; ++mb) {
            float o[C::NP];
            tmem_load<C::NP>(tmem + tlane + C::O_COL + C::NP * mb, o);
#pragma unroll
            for (int r = 0; r < C::PT * C::NQ; ++r) o[r] *= alpha[r % C::NQ];
#pragma unroll
            for (int j = 0; j < C::NP; j += 16) tmem_st16(tmem + tlane + C::O_COL + C::NP * mb + j, o + j);
          }
          tmem_st_wait();
        }
      }
      float w[C::NQ];
#pragma unroll
      for (int r = 0; r < C::NQ; ++r) {
        const float ref = (m_use[r] == kNegInf ? 0.f : m_use[r]) - kBias;
        w[r] = exp2f(t[r] - ref);
        l_part[r] += C::KV8 ? exp2f(sc[r] - ref) : w[r];
      }

      // P(i) -> buffer i % 2; its last reader, P.V(i - 2), must be done
      if (i >= 2) mbar_wait(pv_done + 8 * (i & 1), ((i - 2) >> 1) & 1, failed);
      if (tq == 0) edge[i & 1] = clear;
      unsigned char* pbuf = smem + C::OFF_P + (i & 1) * C::P_BYTES;
      if constexpr (C::KV8) {
#pragma unroll
        for (int r = 0; r < C::NQ; r += 2) {
          float2 x = make_float2(w[r], w[r + 1]);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const uint16_t code = next_term(x);
            const int n = j * C::NQ + r;
            pbuf[swizzled<128>(n, pl >> 4) + (pl & 15)] = static_cast<unsigned char>(code & 0xff);
            pbuf[swizzled<128>(n + 1, pl >> 4) + (pl & 15)] = static_cast<unsigned char>(code >> 8);
          }
        }
      } else {
        unsigned char* half = pbuf + (pl >> 6) * C::NP * 128;
        const int piece = (pl & 63) >> 3, in = (pl & 7) * 2;
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) {
          const uint16_t hi = f32_to_bf16_bits(w[r]);
          const uint16_t lo16 = f32_to_bf16_bits(w[r] - bf16_bits_to_f32(hi));
          *reinterpret_cast<uint16_t*>(half + swizzled<128>(r, piece) + in) = hi;
          *reinterpret_cast<uint16_t*>(half + swizzled<128>(C::NQ + r, piece) + in) = lo16;
        }
      }
      fence_proxy_async_smem();  // P -> the tensor cores' view of shared memory
      tc_fence_before();
      mbar_arrive(p_ready + 8 * (i & 1));

      // A position that takes no part has weight 0, but its V row may hold
      // anything, NaN too: it is cleared before the MMAs read the slot.
      if (clear) {
        for (int p = 0; p < C::NB; ++p) {
          const int e = C::seq_v(i, p, nxt.ok), slot = e % C::RING;
          mbar_wait(full + 8 * slot, (e / C::RING) & 1, failed);
          if (dead_row) {
            for (int ch = 0; ch < C::CH; ++ch)
              for (int x = 0; x < C::SW; x += 16)
                *reinterpret_cast<uint4*>(smem + slot * C::SLOT + ch * C::CHUNK + pl * C::SW + x) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          mbar_arrive(v_clean + 8 * ((i & 1) * C::NB + p));
        }
      }

      if (cur.last) {
        // ---- epilogue: the row sums, then this thread's dim of each block of dims
        float* rs = red + 2 * C::NQ * kSoftWarps;
        const float lsum = rowreduce<C::NQ>(l_part, lane, AddOp());
        named_bar_sync(1, kSoft);  // the last segment's sums have been read
        if (lane % kPer == 0) rs[(lane / kPer) * kSoftWarps + sw] = lsum;
        named_bar_sync(1, kSoft);
        float L[C::NQ];
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) {
          const float4 t4 = *reinterpret_cast<const float4*>(rs + r * kSoftWarps);
          L[r] = (t4.x + t4.y) + (t4.z + t4.w);  // fixed order
        }
        const bool direct = cur.begins && cur.ends;
        const int slot = 2 * c + (cur.begins ? 1 : 0);
        mbar_wait(pv_done + 8 * (i & 1), (i >> 1) & 1, failed);
        tc_fence_after();
#pragma unroll
        for (int mb = 0; mb < C::NB; ++mb) {
          float o[C::NP];
          tmem_load<C::NP>(tmem + tlane + C::O_COL + C::NP * mb, o);
          const int d = mb * 128 + pl;  // O^T lanes are head dims
          if (pl < C::DB) {
#pragma unroll
            for (int r = 0; r < C::NQ; ++r) {
              if (r >= G) break;
              const float x = C::KV8 ? o[r] + (o[C::NQ + r] + o[(C::PT - 1) * C::NQ + r] * 0.0625f) * 0.0625f
                                     : o[r] + o[C::NQ + r];
              if (direct) {
                const size_t at = (static_cast<size_t>(cur.b) * a.NH + static_cast<size_t>(cur.kvh) * G + r) * C::HS + d;
                const float y = L[r] == 0.f ? 0.f : x / L[r];
                a.out[at] = f32_to_bf16_bits(y);
                if (a.out_f32) a.out_f32[at] = y;
              } else {
                a.ws_o[(static_cast<size_t>(slot) * G + r) * C::HS + d] = x;
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(o_free);  // the next segment may use O
        if (!direct && tq < G) {
          float mr = m_use[0], lr = L[0];
#pragma unroll
          for (int r = 1; r < C::NQ; ++r)
            if (r == tq) {
              mr = m_use[r];
              lr = L[r];
            }
          reinterpret_cast<float2*>(a.ws_ml)[static_cast<size_t>(slot) * G + tq] = make_float2(mr, lr);
        }
        if (!nxt.ok && tq == 0) {
          Cut cut{cur.b, cur.kvh, -1, -1};
          if (!cur.ends) {
            const Band d = band_of_seq(a, lens, cur.b);
            const long long u0 = walk.off + static_cast<long long>(cur.kvh) * d.granules;
            cut.c0 = static_cast<int>(u0 / per);
            cut.c1 = static_cast<int>((u0 + d.granules - 1) / per);
          }
          cuts[c] = cut;
        }
      }
      cur = nxt;
      page = next_page;
      ksvs = next_ksvs;
      nxt = after;
      next_page = after_page;
      ++i;
    }
  }

  // release the tensor memory once every warp is done with it
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// ------------------------------------------------------------------- the merge

constexpr int kMergeThreads = 256;

// A unit that lies in the shares c0 .. c1 left a partial in each. Block c in
// [c0, c1) takes its part of the unit's G * HS outputs: one item is four dims
// of a row, whose partials are summed by several threads and then in fixed
// order.
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedArgs a) {
  __shared__ float4 acc[kMergeThreads];
  extern __shared__ float factor[];  // [rows of this block][parts]
  __shared__ float inv[16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Cut cut = reinterpret_cast<const Cut*>(a.cuts)[c];
  if (cut.c0 < 0) return;
  const int G = a.NH / a.NKV, row_items = a.HS / 4, items = G * row_items;
  const int helpers = cut.c1 - cut.c0, parts = helpers + 1;
  const int each = (items + helpers - 1) / helpers;
  const int i0 = (c - cut.c0) * each, i1 = min(items, i0 + each);
  if (i0 >= i1) return;
  const int r0 = i0 / row_items, r1 = (i1 - 1) / row_items;
  // the share c0 holds the unit's beginning, the others continue it
  auto slot_of = [&](int part) { return 2 * (cut.c0 + part) + (part == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml);
  for (int r = r0 + warp; r <= r1; r += kMergeThreads / 32) {
    float m = kNegInf;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, ml[static_cast<size_t>(slot_of(p)) * G + r].x);
    for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float2 x = ml[static_cast<size_t>(slot_of(p)) * G + r];
      // a part whose reference is -inf holds sums that belong to 2^0 (its
      // weights are 0, or NaN, which has to show)
      const float f = x.x == kNegInf ? (x.y == 0.f ? 0.f : x.y) : exp2f(x.x - m);
      factor[(r - r0) * parts + p] = f;
      l += f * x.y;
    }
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    if (lane == 0) inv[r] = l;
  }
  __syncthreads();
  for (int base = i0; base < i1; base += kMergeThreads) {
    const int n = min(kMergeThreads, i1 - base);  // items of this turn
    const int groups = kMergeThreads / n;         // threads of an item
    const int item = base + tid % n, g = tid / n;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const int r = item / row_items, d = item % row_items;
    if (g < groups) {
      const float* f = factor + (r - r0) * parts;
#pragma unroll 8
      for (int p = g; p < parts; p += groups) {
        const float4 x = reinterpret_cast<const float4*>(a.ws_o)[(static_cast<size_t>(slot_of(p)) * G + r) * row_items + d];
        const float w = f[p];
        s.x += w * x.x;
        s.y += w * x.y;
        s.z += w * x.z;
        s.w += w * x.w;
      }
      acc[tid] = s;
    }
    __syncthreads();
    if (g == 0) {
      for (int j = 1; j < groups; ++j) {
        const float4 x = acc[j * n + tid];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
      }
      const float l = inv[r];
      const float4 y = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(s.x / l, s.y / l, s.z / l, s.w / l);
      const size_t at = (static_cast<size_t>(cut.b) * a.NH + static_cast<size_t>(cut.kvh) * G + r) * a.HS + 4 * d;
      const uint32_t lo = f32_to_bf16_bits(y.x) | (static_cast<uint32_t>(f32_to_bf16_bits(y.y)) << 16);
      const uint32_t hi = f32_to_bf16_bits(y.z) | (static_cast<uint32_t>(f32_to_bf16_bits(y.w)) << 16);
      *reinterpret_cast<uint2*>(a.out + at) = make_uint2(lo, hi);
      if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + at) = y;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ the launch

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// A pool as a 3-D tensor (head dim; head and slot; page), read in boxes of one
// swizzle width x `box_rows` rows of one page.
bool encode_pool(CUtensorMap* m, const void* pool, const PagedArgs& a, int sw_bytes) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int eb = a.kv8 ? 1 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.HS), static_cast<cuuint64_t>(a.NKV) * a.P,
                              static_cast<cuuint64_t>(a.num_pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.HS) * eb, static_cast<cuuint64_t>(a.NKV) * a.P * a.HS * eb};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(sw_bytes / eb), static_cast<cuuint32_t>(std::min(a.P, 32)), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, a.kv8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             sw_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_cfg(const PagedArgs& a, cudaStream_t stream) {
  Maps maps;
  if (!encode_pool(&maps.k, a.k, a, C::SW) || !encode_pool(&maps.v, a.v, a, C::SW)) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> attr_done{0};  // bit d: attribute set on device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0 || (attr_done.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(paged_attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<C>, maps, a);
  if (e != cudaSuccess || a.blocks < 2) return e;
  cfg.gridDim = dim3(a.blocks - 1);  // the last share ends where the last unit does
  cfg.blockDim = dim3(kMergeThreads);
  // h helpers and h + 1 parts: (G / h + 2) * (h + 1) <= 2 G + 2 h + 2 factors
  cfg.dynamicSmemBytes = static_cast<size_t>(2 * (a.NH / a.NKV) + 2 * a.blocks + 2) * sizeof(float);
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel, a);
}

template <int HS, bool KV8>
cudaError_t launch_group(const PagedArgs& a, cudaStream_t stream) {
  return a.NH / a.NKV <= 4 ? launch_cfg<Cfg<HS, KV8, 4>>(a, stream) : launch_cfg<Cfg<HS, KV8, 16>>(a, stream);
}

template <bool KV8>
cudaError_t launch_hs(const PagedArgs& a, cudaStream_t stream) {
  switch (a.HS) {
    case 64: return launch_group<64, KV8>(a, stream);
    case 128: return launch_group<128, KV8>(a, stream);
    case 256: return launch_group<256, KV8>(a, stream);
    default: return launch_group<512, KV8>(a, stream);
  }
}

}  // namespace

cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream) {
  return a.kv8 ? launch_hs<true>(a, stream) : launch_hs<false>(a, stream);
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
