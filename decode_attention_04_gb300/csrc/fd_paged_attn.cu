// Single-token attention over a KV cache kept in pages (fd_paged_attn.h), on the
// fifth-generation tensor cores: softmax((q K^T) scale) V with one query token a
// sequence, K and V bf16 or E4M3 with a scale for each page and head.
//
// Work. The live bands of all (sequence, KV head) units lie one behind the
// other in granules of 32 positions, each behind a gap of `min_share` granules
// that stands for what beginning and ending a band costs a block (about as
// much as copying 64 KB; without it the block that had the eight heads of a
// short sequence held up a ragged batch by a fifth). Block c of C takes the places [c, c + 1)
// * ceil(total / C). So every SM has the same work whatever the lengths are,
// in one wave, and a block leaves at most two partials: of a band that began
// before its share and of one that goes on behind it. A band inside one share
// is written to the output directly.
//
// A block, per tile of 128 positions (a share's part of one band is a segment):
//   * Two warps each for K and V fill rings of shared-memory slots (one slot: the
//     tile's 128 positions x 128 head dims) by TMA, a box of one page's rows
//     (32 at most) and 128 bytes each; a lane looks up and copies a box. A box
//     costs its warp about 70 cycles, a slot 200 more: one warp for both tensors
//     fell short of the rate of HBM with pages of 16 (ragged batch 161 us, a warp
//     each 117).
//   * One warp issues S^T (positions x query rows) = K Q^T, one O^T (dims x
//     query rows) += V^T P^T, accumulators in tensor memory. With K as the 128-row operand the
//     tensor cores read every code once, as it lies in the cache: nothing is
//     widened. A warp for both products was the bottleneck: a wait that finds
//     its barrier complete takes 100 cycles, the MMAs of a tile less.
//   * Two groups of four warps turn scores into weights, a position a
//     thread: the groups take the tiles in turn, each with an accumulator, a running
//     maximum and sums of its own, which are joined at the segment's end.
//   * One warp brings the query rows of the next segments.
//   The softmax groups take registers over from the other warps.
//
// E4M3 products are exact but for the other operand, which enters as a sum of
// E4M3 terms, each in MMA columns of its own, term i scaled by 16^i so that it
// has E4M3's full range: q = q0 + q1 / 16 + q2 / 256 (bf16 has 8 significant bits, so elements down to 2^-17 of the row's
// largest are exact and no other is off by more than 2^-25 of it; head dim 512 with 16 rows has two terms, 2^-13 and
// 2^-21: a third takes 16 KB from the ring there, 4 x 131072 MQA 96.4 -> 97.8 us, 32768 positions 20.4 -> 21.5),
// w = w0 + w1 / 16 + ... + w5 / 16^5 (24 bits, as many as the sum has, and nothing is dropped above 2^-30: with three
// terms weights below 2^-18 were, which in a long band are the output where the largest weight's value is
// small). The columns are added in fp32 at the end. 96 columns
// instead of 16 cost the tensor cores nothing here: an MMA takes as long as reading its
// 128-row operand. Head dim 512 with 16 rows has tensor memory for 48 columns: the terms go there in pairs, both
// unscaled in one column, by two MMAs one behind the other, pairs 256 apart (nothing is dropped above 2^-26).
// bf16 takes q as it is and w = w0 + w1 + w2 (24 bits).
//
// Scales. K's multiplies the score. V's multiplies the weight, in units of 2^vref, vref the exponent of the
// largest V scale that the group has met in the segment: w_p = 2^(s_p log2(e) - m) * (vs / 2^vref), so that w fits
// E4M3 whatever the scales are, and the output is multiplied by 2^vref at the end. The maximum m and the row's sum
// l = sum 2^(s_p log2(e) - m) do not know V's scales: a block whose scale is 0 counts in l as any other does.

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
#include "fd_tcgen05.cuh"

// ------------------------------------------------------------- PTX helpers

// 3-D TMA tile load (x = head dim, y = head and slot of a page, z = page).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
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

// The same without a swizzle, MN-major: 16 bytes of a row, rows 16 bytes apart; LBO is the distance between 8-row groups
// along K, SBO between column blocks of 16 bytes.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((8 * 16) >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46);
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

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// Waits for a barrier of each active lane (bounded, as mbar_wait): one round
// trip for all of them.
__device__ __forceinline__ void wait_lanes(uint32_t bar, uint32_t parity, bool active, bool& failed) {
  if (active) mbar_wait(bar, parity, failed);
  failed = __any_sync(0xffffffffu, failed);
  __syncwarp();
}

// A wait of a whole warp. Lanes leave mbar_wait one by one: a lane that ran
// ahead could let the barrier pass two phases before the last one looked, which
// then would wait for ever; and tcgen05.ld wants the warp in step.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, bool& failed) {
  mbar_wait(bar, parity, failed);
  __syncwarp();
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------- the division of work

constexpr int kTile = 128;      // positions per tile: the M of the score MMA
constexpr int kGranule = 32;    // positions; the plan's granule
constexpr int kLenCache = 1024; // lengths kept in shared memory when there are no more sequences
constexpr int kWarpSeqs = 128;  // a warp finds its share by itself when there are no more sequences

struct Band {
  unsigned lo;
  int len, granules;  // live positions [lo, len), counted in granules from floor(lo / 32)
};

__device__ __forceinline__ int clamp_len(const PagedArgs& a, int len) {
  return min(max(len, 0), a.max_pages * a.P);
}

__device__ __forceinline__ Band band_from(const PagedArgs& a, int len) {
  Band d;
  d.len = len;
  d.lo = a.window > 0 ? max(0, len - a.window) : 0u;
  d.granules = len > 0 ? static_cast<int>((len - 1u) / kGranule - d.lo / kGranule + 1) : 0;
  return d;
}

// A share's part of one unit's band.
struct Tile {
  int b, kvh;
  int pos;         // first position (a multiple of 32)
  int end;         // positions [max(pos, lo), min(pos + 128, end)) are live in the segment
  int lo;
  int seg;         // number of the segment in this block
  int j, n;        // tile j of the segment's n
  bool begins, ends;   // the segment holds the band's first / last granule
  bool ok;
};

// Walks a block's tiles in order.
struct Walk {
  long long left;  // places of the share that are still to come
  int kvh, g0;     // where the next segment begins: head, place of the band (gap, then granules)
  Band d;          // of sequence t.b
  Tile t;
};

__device__ __forceinline__ Band band_of_seq(const PagedArgs& a, const int* cache, int b) {
  return band_from(a, a.B <= kLenCache ? cache[b] : clamp_len(a, a.lens[b]));
}

// Places of one unit in the stream; none where there is no position.
__device__ __forceinline__ int places(const PagedArgs& a, const Band& d) {
  return d.granules > 0 ? d.granules + a.min_share : 0;
}

__device__ __forceinline__ void next_tile(const PagedArgs& a, const int* cache, Walk& w) {
  Tile& t = w.t;
  if (t.j + 1 < t.n) {
    t.pos += kTile;
    t.j += 1;
    return;
  }
  if (w.left <= 0) {
    t.ok = false;
    t.n = 0;
    return;
  }
  int b = t.b;
  while (w.g0 >= places(a, w.d)) {  // the band is done: the next head, or the next sequence that has one
    w.g0 = 0;
    if (++w.kvh >= a.NKV || w.d.granules == 0) {
      w.kvh = 0;
      w.d = band_of_seq(a, cache, ++b);
    }
  }
  if (w.g0 < a.min_share) {  // the gap
    const int skip = static_cast<int>(min(static_cast<long long>(a.min_share - w.g0), w.left));
    w.left -= skip;
    w.g0 += skip;
    if (w.left <= 0) {
      t.ok = false;
      t.n = 0;
      return;
    }
  }
  const int take = static_cast<int>(min(static_cast<long long>(places(a, w.d) - w.g0), w.left));
  w.left -= take;
  t.b = b;
  t.seg += 1;
  t.kvh = w.kvh;
  t.lo = w.d.lo;
  t.pos = (w.d.lo / kGranule + w.g0 - a.min_share) * kGranule;
  t.begins = w.g0 == a.min_share;
  w.g0 += take;
  t.ends = w.g0 == places(a, w.d);
  t.end = t.ends ? w.d.len : t.pos + take * kGranule;
  t.j = 0;
  t.n = (t.end - t.pos + kTile - 1) / kTile;
  t.ok = true;
}

// --------------------------------------------------------------------- shapes

constexpr int kSoftWarps = 4;  // of a softmax group: one TMEM lane quarter each
constexpr int kSoft = kSoftWarps * 32;
// Warps, by fours (warpgroups): the first copy warps and the MMA warps; the two
// softmax groups; the query rows and the second copy warps.
constexpr int W_K = 0, W_QK = 1, W_PV = 2, W_V = 3, W_SOFT0 = 4, W_Q = 12, W_K2 = 13, W_V2 = 14;
constexpr int kThreads = 16 * 32;
// Registers a thread of each warpgroup: 72 + 2 * 184 + 64 <= 4 * 128, what the block is launched with.
constexpr int kRegsIssue = 72, kRegsSoft = 184, kRegsHelp = 64;
static_assert(kRegsIssue + 2 * kRegsSoft + kRegsHelp <= 4 * (65536 / kThreads), "registers of the launch");
constexpr int kQRing = 8;      // segments whose query multipliers are kept
constexpr int BAR_GROUP = 1, BAR_BOTH = 3;  // named barriers: of a softmax group (two), of both

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
  static constexpr bool WIDE = KV8 && HS * NQ > 4096;  // head dim 512, 16 rows: the least shared and tensor memory a term
  static constexpr int QT = !KV8 ? 1 : WIDE ? 2 : 3;   // terms of q
  static constexpr int PT = KV8 ? 6 : 3;               // terms of a weight
  static constexpr int PP = WIDE ? 2 : 1;              // of them in a column
  static constexpr int NS = round16(QT * NQ);          // columns of S
  static constexpr int NP = round16(PT / PP * NQ);     // columns of O
  static constexpr int COLS = pow2_cols(2 * NS + 2 * NB * NP);
  static constexpr int O_COL = 2 * NS;
  static constexpr int Q_BYTES = NB * CH * NS * SW;
  static constexpr int P_BYTES = PP * NP * kTile * EB;
  static constexpr int RED_BYTES = (2 * 11 + 4) * NQ * 4 + 64;
  static constexpr int Q_STRIDE = (Q_BYTES + 1023) / 1024 * 1024;
  static constexpr int RING_ROOM = 227 * 1024 - 2 * Q_STRIDE - 2 * P_BYTES - RED_BYTES - kLenCache * 4 - 2048;
  static constexpr int RING = RING_ROOM / SLOT < 24 ? RING_ROOM / SLOT : 24;  // slots: all the shared memory there is
  static constexpr int OFF_Q = RING * SLOT;
  static constexpr int OFF_P = OFF_Q + 2 * Q_STRIDE;
  // f32, of each group 11 NQ, of both 4 NQ: the groups' statistics; int: exponents of V's scales
  static constexpr int OFF_RED = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_QMUL = OFF_RED + RED_BYTES;  // f32 [kQRing][16]
  static constexpr int OFF_LEN = OFF_QMUL + kQRing * 16 * 4;
  static constexpr int OFF_BAR = OFF_LEN + kLenCache * 4;
  // full[RING], empty[RING], s_full[2], s_free[2], p_ready[2], pv_done[2], q_ready[2], q_free[2], o_free[2], mma_done[2],
  // v_clean[2][NB], v_here[2][NB]; the pairs by the parity of a tile (its group) or, for q, of a segment
  static constexpr int NBAR = 2 * RING + 16 + 4 * NB;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tensor memory address; share; edge[2]
  static constexpr int SMEM = OFF_MISC + 64 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * NS + 2 * NB * NP <= 512, "tensor memory");
  static_assert(Q_STRIDE % 1024 == 0, "swizzle atoms are aligned");
  static_assert(OFF_BAR % 8 == 0, "barriers");
  static constexpr int RK = RING / 2, RV = RING - RK;  // K's slots, then V's
  static_assert(RK >= 2, "two slots of each of K and V");
  // Instruction descriptor: D f32; A and B E4M3 (0) or bf16 (1 in bits 7 and
  // 10); bits 15 and 16: A and B are MN-major; N / 8 at 17, M / 16 at 24.
  static constexpr uint32_t IDESC_QK = (1u << 4) | (KV8 ? 0u : (1u << 7) | (1u << 10)) |
                                       (static_cast<uint32_t>(NS >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
  static constexpr uint32_t IDESC_PV = (1u << 4) | (KV8 ? 0u : (1u << 7) | (1u << 10)) | (3u << 15) |
                                       (static_cast<uint32_t>(NP >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
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

// x = c0 + c1 / 16 + c2 / 256 + ... (by = 16): the next E4M3 term of a pair; x becomes
// what is left, times `by`. x is at most 448 in size.
__device__ __forceinline__ uint16_t next_term(float2& x, float by) {
  const uint16_t c = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
  const float2 y = e4m3x2_to_f32(c);
  x.x = (x.x - y.x) * by;
  x.y = (x.y - y.y) * by;
  return c;
}

// The same of a pair of fp16 values, exactly: what a term leaves is a multiple of x's last place.
__device__ __forceinline__ uint16_t next_term(__half2& x, float by) {
  const uint16_t c = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
  x = __hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
  if (by != 1.f) x = __hmul2(x, __float2half2_rn(by));
  return c;
}

// Six terms of a pair of weights of at most 2^8, PP of them to a column (the columns 16^PP apart). In fp16 where that
// holds what is left (its first 11 bits, after four terms the rest): half as many instructions as in fp32.
template <int PP>
__device__ __forceinline__ void six_terms(float2 w, uint16_t (&c)[6]) {
  // behind the terms that end a column, and behind the others
  constexpr float kLast = PP == 1 ? 16.f : 256.f, kFirst = PP == 1 ? 16.f : 1.f;
  __half2 x = __floats2half2_rn(w.x, w.y);
  const float2 hi = __half22float2(x);
  c[0] = next_term(x, kFirst);
  c[1] = next_term(x, kLast);
  c[2] = next_term(x, kFirst);
  const float2 left = __half22float2(x);
  constexpr float kScale = PP == 1 ? 4096.f : 256.f;  // of what is left by now
  float2 z = make_float2(fmaf(w.x - hi.x, kScale, left.x), fmaf(w.y - hi.y, kScale, left.y));
  c[3] = next_term(z, kLast);
  x = __floats2half2_rn(z.x, z.y);
  c[4] = next_term(x, kFirst);
  c[5] = next_term(x, kLast);
}

struct Maps {
  CUtensorMap k, v;
};

// 2^n for n <= 127 (0 below 2^-126).
__device__ __forceinline__ float pow2_of(int n) {
  return n < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}

// The exponent of a scale, of zero kNoScale.
constexpr int kNoScale = -150;
__device__ __forceinline__ int exponent_of(float s) {
  const uint32_t u = __float_as_uint(s) & 0x7fffffffu;
  return u >= 0x00800000u ? static_cast<int>(u >> 23) - 127 : 31 - __clz(u) - 149;
}

// Which units a block's share breaks: written for the merge.
struct Cut {
  int b, kvh;
  int c0, c1;  // the unit lies in the shares c0 .. c1; c0 < 0: the share ends where a unit does
};

// The smallest power of the running reference that is moved: 2^(s - m) is at most 2^(kLazy + kBias). E4M3: that is
// 2^7, and V's scale in units of 2^vref is below 2, which keeps weights within E4M3's 448. A higher bias leaves
// smaller weights above what the terms drop, a lower one moves the reference less often: terms with a column each drop
// less and take the lower one (a move at 2^3 / 2^4 / 2^5: ragged batch E4M3 107 / 106 / 105 us, 4 x 131072 MQA 97.7 /
// 97.6 / 97.6, both before the issue loops were rolled).
constexpr float kTop8 = 7.f, kLazy8 = 5.f, kLazy8Shared = 3.f;
// bf16: 2^(s - m) is at most 2^8, and enters the product with V times 2^-8: no value that is finite in V leaves fp32
// where the largest weight meets it.
constexpr float kLazy16 = 8.f, kBias16 = 0.f, kUnit16 = 0x1p-8f;

template <class C>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ Maps maps, const PagedArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  const int c = blockIdx.x;
  const int G = a.NH / a.NKV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int page_shift = 31 - __clz(a.P);

  const uint32_t bar0 = base + C::OFF_BAR;
  const uint32_t full = bar0, empty = full + 8 * C::RING;
  const uint32_t s_full = empty + 8 * C::RING, s_free = s_full + 16, p_ready = s_free + 16, pv_done = p_ready + 16;
  const uint32_t q_ready = pv_done + 16, q_free = q_ready + 16, o_free = q_free + 16, mma_done = o_free + 16;
  const uint32_t v_clean = mma_done + 16, v_here = v_clean + 16 * C::NB;
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* qmul = reinterpret_cast<float*>(smem + C::OFF_QMUL);
  int* lens = reinterpret_cast<int*>(smem + C::OFF_LEN);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* share_at = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);  // where the share begins: sequence, head, granule
  volatile int* edge = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 32);  // of tile i: V has rows to clear

  // Set-up that reads no input, overlapping the previous kernel's tail.
  if (tid == 0) {
    for (int k = 0; k < C::RING; ++k) {
      mbar_init(full + 8 * k, 2);  // both copy warps, and the bytes
      mbar_init(empty + 8 * k, 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(s_full + 8 * j, 1);
      mbar_init(s_free + 8 * j, kSoft);
      mbar_init(p_ready + 8 * j, kSoft);
      mbar_init(pv_done + 8 * j, 1);
      mbar_init(q_ready + 8 * j, 1);
      mbar_init(q_free + 8 * j, 1);
      mbar_init(o_free + 8 * j, 2 * kSoft);
    }
    for (int j = 0; j < 2 * C::NB; ++j) {
      mbar_init(v_clean + 8 * j, kSoft);
      mbar_init(v_here + 8 * j, 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(mma_done + 8, 1);
    fence_mbar_init();
    prefetch_tensor_map(&maps.k);
    prefetch_tensor_map(&maps.v);
  }
  if (warp == W_QK) {
    tmem_alloc(base + C::OFF_MISC, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_dependency_wait();
  grid_launch_dependents();

  // This block's share of the places, and where it begins.
  long long per, total;
  Walk walk;
  walk.t.ok = false;
  walk.t.seg = -1;
  walk.t.j = walk.t.n = 0;
  walk.t.b = walk.kvh = walk.g0 = 0;
  auto shares = [&](long long of_a_head) {  // places of one head of every sequence
    total = of_a_head * a.NKV;
    per = total <= 0x7fff0000ll ? static_cast<int>(total + a.blocks - 1) / a.blocks : (total + a.blocks - 1) / a.blocks;
    per = max(per, static_cast<long long>(a.min_share));
    walk.left = min(per, total - per * c);
  };
  // sequence b, whose units have x places each and begin at place off of the stream, holds the share's first
  auto begin_at = [&](int b, long long off, int x) {
    const long long in = per * c - off;
    walk.t.b = b;
    if (in <= 0x7fffffffll) {
      walk.kvh = static_cast<int>(in) / x;
      walk.g0 = static_cast<int>(in) % x;
    } else {
      walk.kvh = static_cast<int>(in / x);
      walk.g0 = static_cast<int>(in % x);
    }
  };
  if (a.B <= kWarpSeqs) {
    // Every warp by itself, without a barrier, 32 sequences a turn (a turn is
    // little code: fetching it is most of what it costs). A head's places are
    // below 2^31 (checked on the host).
    unsigned flags = 0;
    int sum = 0, x = 0, upto = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int raw_len = b < a.B ? a.lens[b] : 0, len = clamp_len(a, raw_len);
      if (raw_len < 0) flags |= FD_DEVERR_LEN_NEGATIVE;
      if (raw_len > len) flags |= FD_DEVERR_LEN_CLAMPED;
      if (b < a.B) lens[b] = len;  // each warp writes the same, and reads its own
      x = places(a, band_from(a, len));
      upto = x;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, i);
        if (lane >= i) upto += y;
      }
      upto += sum;
      sum = __shfl_sync(0xffffffffu, upto, 31);
    }
    if (c == 0 && warp == 0 && flags) atomicOr(&g_device_error, flags);
    shares(sum);
    // the sequence that holds the share's first place, from the last turn backwards
    const long long start = per * c;
#pragma unroll 1
    for (int b0 = (a.B - 1) & ~31; walk.left > 0; b0 -= 32) {
      const long long off = static_cast<long long>(upto - x) * a.NKV;
      const unsigned who = __ballot_sync(0xffffffffu, x > 0 && off <= start);
      if (who) {  // the last one that begins at or before it
        const int src = 31 - __clz(who);
        begin_at(b0 + src, __shfl_sync(0xffffffffu, off, src), __shfl_sync(0xffffffffu, x, src));
        break;
      }
      // a turn earlier: its places end where this one's begin
      const int end = __shfl_sync(0xffffffffu, upto - x, 0);
      x = places(a, band_from(a, lens[b0 - 32 + lane]));
      upto = x;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, i);
        if (lane >= i) upto += y;
      }
      upto += end - __shfl_sync(0xffffffffu, upto, 31);
    }
    __syncwarp();
  } else {
    long long* sums = reinterpret_cast<long long*>(smem + C::OFF_RED);  // [kThreads / 32]
    long long mine = 0;
    unsigned flags = 0;
    for (int b = tid; b < a.B; b += kThreads) {
      const int raw_len = a.lens[b], len = clamp_len(a, raw_len);
      if (raw_len < 0) flags |= FD_DEVERR_LEN_NEGATIVE;
      if (raw_len > len) flags |= FD_DEVERR_LEN_CLAMPED;
      if (a.B <= kLenCache) lens[b] = len;
      mine += places(a, band_from(a, len));
    }
    if (c == 0 && flags) atomicOr(&g_device_error, flags);
    for (int i = 16; i; i >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, i);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    long long all = 0;
    for (int i = 0; i < kThreads / 32; ++i) all += sums[i];
    shares(all);
    const long long start = per * c;
    long long before = 0;  // places (of one head) of the sequences before this chunk
    for (int b0 = 0; b0 < a.B && start < total; b0 += kThreads) {
      const int b = b0 + tid;
      const int x = b < a.B ? places(a, band_of_seq(a, lens, b)) : 0;
      long long inc = x;
      for (int i = 1; i < 32; i <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, i);
        if (lane >= i) inc += y;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      all = 0;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) inc += sums[i];
        all += sums[i];
      }
      const long long off = (before + inc - x) * a.NKV;
      if (x > 0 && off <= start && start < off + static_cast<long long>(x) * a.NKV) {
        begin_at(b, off, x);
        share_at[0] = walk.t.b;
        share_at[1] = walk.kvh;
        share_at[2] = walk.g0;
      }
      before += all;
      if (start < before * a.NKV) break;
    }
    __syncthreads();
    if (walk.left > 0) {
      walk.t.b = share_at[0];
      walk.kvh = share_at[1];
      walk.g0 = share_at[2];
    }
  }
  if (walk.left > 0) {
    walk.d = band_of_seq(a, lens, walk.t.b);
    next_tile(a, lens, walk);
  }
  const bool work = walk.t.ok;

  Cut* cuts = reinterpret_cast<Cut*>(a.cuts);
  if (!work && tid == 0) cuts[c].c0 = -1;

  bool failed = false;
  int slots_used = 0;  // of the ring of a copy warp

  // Query rows of a segment -> the B operand of its score MMAs: rows of SW bytes, swizzled,
  // term j of row r in row j * NQ + r; rows >= G are zero.
  auto stage_q = [&](const Tile& t, int first, int threads) {
    const int par = t.seg & 1;
    unsigned char* qb = smem + C::OFF_Q + par * C::Q_STRIDE;
    constexpr int EL = 16 / C::EB;           // elements of a 16-byte piece
    constexpr int PIECES = C::HS / EL;       // of a row: a power of two, at most 64
    for (int id = first; (id & ~31) < C::NQ * PIECES; id += threads) {  // whole warps
      const int r = id / PIECES, pc = id % PIECES;
      const bool live = r < G && r < C::NQ;
      const int chunk = pc * 16 / C::SW, piece = (pc * 16 % C::SW) / 16;
      const size_t row = static_cast<size_t>(t.b) * a.NH + static_cast<size_t>(t.kvh) * G + r;
      const uint16_t* src = a.q + row * C::HS + pc * EL;
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
        if (pc == 0 && r < C::NQ)
          qmul[(t.seg & (kQRing - 1)) * 16 + r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
        uint32_t w[C::QT][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 y = make_float2(f[i].x * mul, f[i].y * mul);
          // an infinity would saturate: it has to reach the scores as NaN
          if (ex == 255) {
            y.x = isfinite(y.x) ? y.x : __int_as_float(0x7fffffff);
            y.y = isfinite(y.y) ? y.y : __int_as_float(0x7fffffff);
          }
          __half2 h = __floats2half2_rn(y.x, y.y);  // exact above 2^-17, else to 2^-25
#pragma unroll
          for (int j = 0; j < C::QT; ++j) {
            const uint32_t term = next_term(h, 16.f);
            if (i & 1) w[j][i / 2] |= term << 16;
            else w[j][i / 2] = term;
          }
        }
        if (r < C::NQ) {
#pragma unroll
          for (int j = 0; j < C::QT; ++j)
            *reinterpret_cast<uint4*>(qb + chunk * C::NS * C::SW + swizzled<C::SW>(j * C::NQ + r, piece)) =
                make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
        }
      }
    }
    fence_proxy_async_smem();
  };

  // ---------------------------------------------------------------- copy warps
  auto copy_tiles = [&] {
    const bool is_k = warp == W_K || warp == W_K2;
    const CUtensorMap* map = is_k ? &maps.k : &maps.v;
    const int ring = is_k ? C::RK : C::RV, slot0 = is_k ? 0 : C::RK;
    const int box = min(a.P, 32);           // rows of a copy
    const int half = kTile / box / 2;       // boxes of a tile that are this warp's
    const uint32_t box_bytes = box * C::SW * C::CH;
    const int row = (lane + (warp < W_SOFT0 ? 0 : half)) * box;  // this lane's box in a tile
    // the table's entry for this lane's box in a tile; -1: nothing to copy
    auto page_of = [&](const Tile& t) {
      if (!t.ok || lane >= half || row >= t.end - t.pos || t.pos + row + box <= t.lo) return -1;
      return a.table[static_cast<size_t>(t.b) * a.max_pages + ((t.pos + row) >> page_shift)];
    };
    Tile cur = walk.t;
    int page = page_of(cur);
    int slot = slot0;
    uint32_t turn = 1;  // parity of `empty` that lets this turn of the ring begin: none in the first
    for (int n = 0; cur.ok && n < a.withhold_tile; ++n) {
      next_tile(a, lens, walk);
      const Tile nxt = walk.t;
      const int next_page = page_of(nxt);  // in flight while this tile's copies wait for slots
      const bool there = page >= 0 && page < a.num_pages;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, there)) * box_bytes;
      const int y = cur.kvh * a.P + ((cur.pos + row) & (a.P - 1));
#pragma unroll 1
      for (int p = 0; p < C::NB; ++p) {
        if (slots_used >= ring) warp_wait(empty + 8 * slot, turn, failed);
        const uint32_t fb = full + 8 * slot;
        if (lane == 0) mbar_arrive_expect_tx(fb, bytes);
        __syncwarp();
        if (there) {
#pragma unroll
          for (int ch = 0; ch < C::CH; ++ch)
            tma_load_3d(base + slot * C::SLOT + ch * C::CHUNK + row * C::SW, map, p * C::DB + ch * (C::SW / C::EB), y,
                        page, fb);
        }
        ++slots_used;
        if (++slot == slot0 + ring) {
          slot = slot0;
          turn ^= 1;
        }
      }
      cur = nxt;
      page = next_page;
    }
  };

  // A warpgroup takes its registers in one place, all of its warps together.
  if (!work) {
    // nothing but the rows of empty sequences, below
  } else if (warp < W_SOFT0) {
    regs_dec<kRegsIssue>();
    if (warp == W_K || warp == W_V) {
      copy_tiles();
    } else if (warp == W_QK) {
      // ------------------------------------------------------------ scores: S^T = K Q^T
      // The whole warp in step, one lane issues. The descriptors of a slot differ
      // from those of slot 0 by its address.
      const bool issuer = elect_one();
      const uint64_t k_desc = smem_desc<C::SW>(base, 16);
      const uint64_t q_desc = smem_desc<C::SW>(base + C::OFF_Q, 16);
      int slot = 0;
      uint32_t turn = 0;  // parity of the ring's turn
      for (int i = 0; walk.t.ok; ++i) {
        const int g = i & 1, par = walk.t.seg & 1;
        const bool ends = walk.t.j + 1 == walk.t.n;
        const uint64_t qd = q_desc + par * (C::Q_STRIDE >> 4);
        const uint32_t d = tmem + C::NS * g;
        // the first slot, the S buffer, the segment's query rows: a lane each
        uint32_t bar = full + 8 * slot, want = turn;
        if (lane == 1) bar = s_free + 8 * g, want = ((i >> 1) - 1) & 1;
        if (lane == 2) bar = q_ready + 8 * par, want = (walk.t.seg >> 1) & 1;
        wait_lanes(bar, want, lane == 0 || (lane == 1 && i >= 2) || (lane == 2 && walk.t.j == 0), failed);
#pragma unroll 1
        for (int p = 0; p < C::NB; ++p) {
          if (p > 0) warp_wait(full + 8 * slot, turn, failed);
          tc_fence_after();
          if (issuer) {
            const uint64_t qp = qd + p * ((C::CH * C::NS * C::SW) >> 4);
            const uint64_t kd = k_desc + static_cast<uint32_t>(slot) * (C::SLOT >> 4);
#pragma unroll
            for (int ch = 0; ch < C::CH; ++ch)
#pragma unroll
              for (int kk = 0; kk < C::SW / 32; ++kk)
                umma<C::KV8>(d, kd + ((ch * C::CHUNK + 32 * kk) >> 4),
                             qp + ((ch * C::NS * C::SW + 32 * kk) >> 4), C::IDESC_QK, (p | ch | kk) != 0);
            umma_commit(empty + 8 * slot);
            if (p == C::NB - 1) {
              umma_commit(s_full + 8 * g);
              if (ends) umma_commit(q_free + 8 * par);
            }
          }
          if (++slot == C::RK) {
            slot = 0;
            turn ^= 1;
          }
        }
        next_tile(a, lens, walk);
      }
      // every MMA issued has completed before the tensor memory is released
      if (issuer) umma_commit(mma_done);
      bool dfail = false;
      warp_wait(mma_done, 0, dfail);
    } else if (warp == W_PV) {
      // ------------------------------------------------------------ values: O^T += V^T P^T
      const bool issuer = elect_one();
      const uint64_t v_desc = smem_desc<C::SW>(base, C::CH > 1 ? C::CHUNK : C::SLOT);
      const uint64_t p_desc = smem_desc_plain(base + C::OFF_P, 16 * kTile);
      int slot = C::RK;
      uint32_t turn = 0;
      // bit g, of group g: parity of v_clean's phase, of o_free's, and whether O was used
      uint32_t cleared = 0, o_phase = 0, o_used = 0;
      for (int i = 0; walk.t.ok; ++i) {
        const int g = i & 1;
        const bool takes = walk.t.j < 2;  // the group's first tile of the segment takes O
        // the first slot, the weights, and that the group's segment before has left O: a lane each
        uint32_t bar = full + 8 * slot, want = turn;
        if (lane == 1) bar = p_ready + 8 * g, want = (i >> 1) & 1;
        if (lane == 2) bar = o_free + 8 * g, want = (o_phase >> g) & 1;
        const bool wait_o = takes && ((o_used >> g) & 1);
        wait_lanes(bar, want, lane < 2 || (lane == 2 && wait_o), failed);
        if (wait_o) o_phase ^= 1u << g;
        if (takes) o_used |= 1u << g;
        // read by every lane before one of them issues what lets the group write the next
        const bool clear = __any_sync(0xffffffffu, edge[g] != 0);
        const uint64_t pd = p_desc + g * (C::P_BYTES >> 4);
        const int nk = (min(kTile, walk.t.end - walk.t.pos) + C::KSTEP - 1) / C::KSTEP;
        const uint32_t keep = takes ? 0u : 1u;
#pragma unroll 1
        for (int p = 0; p < C::NB; ++p) {
          if (p > 0) warp_wait(full + 8 * slot, turn, failed);
          if (clear) {  // the group clears rows of the slot first
            if (issuer) mbar_arrive(v_here + 8 * (g * C::NB + p));
            warp_wait(v_clean + 8 * (g * C::NB + p), (cleared >> g) & 1, failed);
          }
          tc_fence_after();
          if (issuer) {
            const uint32_t d = tmem + C::O_COL + C::NP * (g * C::NB + p);
            const uint64_t vd = v_desc + static_cast<uint32_t>(slot) * (C::SLOT >> 4);
            // in loops: the block's code has to fit the instruction cache (unrolled: ragged batch E4M3 104 us, so 98)
#pragma unroll 1
            for (int t = 0; t < C::PP; ++t)
#pragma unroll 1
              for (int kk = 0; kk < nk; ++kk)
                umma<C::KV8>(d, vd + ((kk * C::KSTEP * C::SW) >> 4),
                             pd + ((t * C::NP * kTile * C::EB + kk * C::KSTEP * 16) >> 4), C::IDESC_PV,
                             (t | kk) != 0 ? 1u : keep);
            umma_commit(empty + 8 * slot);
            if (p == C::NB - 1) umma_commit(pv_done + 8 * g);
          }
          if (++slot == C::RING) {
            slot = C::RK;
            turn ^= 1;
          }
        }
        if (clear) cleared ^= 1u << g;
        next_tile(a, lens, walk);
      }
      if (issuer) umma_commit(mma_done + 8);
      bool dfail = false;
      warp_wait(mma_done + 8, 0, dfail);
    }
  } else if (warp >= W_Q) {
    regs_dec<kRegsHelp>();
    if (warp == W_K2 || warp == W_V2) {
      copy_tiles();
    } else if (warp == W_Q) {
      // ------------------------------------------------ query rows, from the second segment on
      for (;;) {
        walk.t.j = walk.t.n;  // on to the next segment
        next_tile(a, lens, walk);
        if (!walk.t.ok) break;
        const int seg = walk.t.seg;
        if (seg >= 2) warp_wait(q_free + 8 * (seg & 1), ((seg - 2) >> 1) & 1, failed);
        stage_q(walk.t, lane, 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready + 8 * (seg & 1));
      }
      // the unit that the share's end cuts, if it does: for the merge
      if (lane == 0) {
        Cut cut{walk.t.b, walk.t.kvh, -1, -1};
        if (!walk.t.ends) {
          // of the band's first granule; a share that ends inside a band is a full one
          const long long u0 = per * (c + 1) - walk.g0 + a.min_share;
          cut.c0 = static_cast<int>(u0 / per);
          cut.c1 = static_cast<int>((u0 + walk.d.granules - 1) / per);
        }
        cuts[c] = cut;
      }
    }
  } else {
    // ---------------------------------------------- softmax / epilogue warps
    regs_inc<kRegsSoft>();
    constexpr float kLazy = !C::KV8 ? kLazy16 : C::PP == 1 ? kLazy8 : kLazy8Shared;
    constexpr float kBias = !C::KV8 ? kBias16 : kTop8 - kLazy;
    const int grp = (warp - W_SOFT0) / kSoftWarps;  // takes the tiles i with i % 2 == grp
    const int sw = (warp - W_SOFT0) % kSoftWarps;
    const int quarter = warp & 3;   // the TMEM lane quarter this warp may access
    const int tq = tid - W_SOFT0 * 32 - grp * kSoft;
    const int pl = quarter * 32 + lane;  // the tile's position whose scores this thread holds
    const uint32_t tlane = static_cast<uint32_t>(quarter * 32) << 16;

    // Of this thread's position: the table's entry, two tiles ahead, and the
    // block's scales, one tile ahead: both are in flight while a tile is worked on. -1: the position takes no part.
    auto entry = [&](const Tile& t) {
      const int pos = t.pos + pl;
      if (!t.ok || pl >= t.end - t.pos || pos < t.lo) return -1;
      return a.table[static_cast<size_t>(t.b) * a.max_pages + (pos >> page_shift)];
    };
    auto scales = [&](const Tile& t, int page) {
      if (!C::KV8 || page < 0 || page >= a.num_pages) return make_float2(0.f, 0.f);
      const size_t at = static_cast<size_t>(page) * a.NKV + t.kvh;
      return make_float2(a.k_scale[at], a.v_scale[at]);
    };

    // Shared memory of the group: [NQ][4] maxima, [NQ][4] sums, [NQ] references, [2][NQ] factors of
    // the accumulators; of both groups: [2][NQ] (reference, sum).
    float* part = red + grp * 11 * C::NQ;
    float* sums = part + 4 * C::NQ;
    float* refs = sums + 4 * C::NQ;
    float* fac = refs + C::NQ;
    float2* stat = reinterpret_cast<float2*>(red + 2 * 11 * C::NQ);
    // exponents of V's scales: the largest of each warp's positions in a tile; of each group's in a segment, and the
    // part of it that the output takes
    int* vtops = reinterpret_cast<int*>(red + 26 * C::NQ) + 4 * grp;
    int* vrefs = reinterpret_cast<int*>(red + 26 * C::NQ) + 8;
    const uint32_t o_cols = tmem + tlane + C::O_COL;

    // This group's tiles: the current one and the next. The look-ups are in
    // flight while the first segment's query rows are brought.
    const Tile first_tile = walk.t;
    if (grp == 1) next_tile(a, lens, walk);
    Tile cur = walk.t;
    int page = entry(cur);
    stage_q(first_tile, tid - W_SOFT0 * 32, 2 * kSoft);
    float2 ksvs = scales(cur, page);
    named_bar_sync(BAR_BOTH, 2 * kSoft);
    if (grp == 0 && tq == 0) mbar_arrive(q_ready);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) next_tile(a, lens, walk);
    Tile nxt = walk.t;
    int next_page = entry(nxt);
    // Per row: the reference (the running maximum less the bias), this thread's share of the sum. A lane
    // also keeps the reference of the row that it ends with in a row reduction.
    constexpr float kNone = -3e38f;  // below every score
    constexpr int kPer = 32 / C::NQ; // lanes that end with the same row
    float ref[C::NQ], l_part[C::NQ];
    float ref_lane = kNone;
    // V's scales: the exponent vref that they are held in units of, 2^-vref as two factors (alone it may not be a
    // float), and the least scale that moves it.
    int vref;
    float vunit[2], vlim;
    auto set_vref = [&](int e) {
      vref = e;
      vunit[0] = pow2_of(-(e >> 1));
      vunit[1] = pow2_of((e >> 1) - e);
      vlim = e == kNoScale ? __uint_as_float(1) : e < 127 ? pow2_of(e + 1) : -kNegInf;
    };
    set_vref(kNoScale);
    int i = grp, seg_seen = -1, cleared = 0;
    while (cur.ok) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) next_tile(a, lens, walk);
      const Tile after = walk.t;
      const int after_page = entry(after);
      const float2 next_ksvs = scales(nxt, next_page);
      const int u = i >> 1;  // number of the tile within the group
      if (cur.seg != seg_seen) {
        seg_seen = cur.seg;
        ref_lane = kNone;
        set_vref(kNoScale);
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) {
          ref[r] = kNone;
          l_part[r] = 0.f;
        }
      }
      const bool live = page >= 0 && page < a.num_pages;
      const int rows = (min(kTile, cur.end - cur.pos) + C::KSTEP - 1) / C::KSTEP * C::KSTEP;  // that P.V reads
      const bool dead_row = !live && pl < rows;

      warp_wait(s_full + 8 * grp, u & 1, failed);
      tc_fence_after();
      float s[C::NS];
      tmem_load<C::NS>(tmem + tlane + C::NS * grp, s);
      tc_fence_before();
      mbar_arrive(s_free + 8 * grp);

      // the segment's multipliers were in place before its score MMAs were issued
      float sc[C::NQ];  // log2 of the weight
      if constexpr (C::KV8) {
        const float4* qm = reinterpret_cast<const float4*>(qmul + (cur.seg & (kQRing - 1)) * 16);
#pragma unroll
        for (int r = 0; r < C::NQ; r += 4) {
          const float4 m = qm[r / 4];
          const float mul[4] = {ksvs.x * m.x, ksvs.x * m.y, ksvs.x * m.z, ksvs.x * m.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float low = s[C::NQ + r + j];
            if constexpr (C::QT > 2) low += s[2 * C::NQ + r + j] * 0.0625f;
            sc[r + j] = live ? (s[r + j] + low * 0.0625f) * mul[j] : kNegInf;
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) sc[r] = live ? s[r] * a.scale_log2 : kNegInf;
      }
      // The tile's row maxima. Most tiles move no reference and have every row live: one
      // barrier tells the group so.
      const float wmax = rowreduce<C::NQ>(sc, lane, MaxOp());
      bool clear = false;
      if (named_bar_or(BAR_GROUP + grp, kSoft,
                       dead_row || wmax > ref_lane + (kLazy + kBias) || (C::KV8 && ksvs.y >= vlim))) {
        if (dead_row && cur.pos + pl >= cur.lo && cur.pos + pl < cur.end) atomicOr(&g_device_error, FD_DEVERR_PAGE_ID);
        if (lane % kPer == 0) part[(lane / kPer) * kSoftWarps + sw] = wmax;
        if constexpr (C::KV8) {
          const int vtop = __reduce_max_sync(0xffffffffu, exponent_of(ksvs.y));
          if (lane == 0) vtops[sw] = vtop;
        }
        clear = named_bar_or(BAR_GROUP + grp, kSoft, dead_row);
        auto row_max = [&](int r) {
          const float4 t4 = *reinterpret_cast<const float4*>(part + r * kSoftWarps);
          return fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
        };
        // every thread takes the same decisions from the same shared values
        const float ml = row_max(lane / kPer);
        if (ml > ref_lane + (kLazy + kBias)) ref_lane = ml - kBias;  // false for -inf and NaN
        float alpha[C::NQ];
        float valpha = 1.f;  // of the accumulators beside alpha
        bool resc = false;
        if constexpr (C::KV8) {
          const int4 v4 = *reinterpret_cast<const int4*>(vtops);
          const int to = max(max(vref, max(v4.x, v4.y)), max(v4.z, v4.w));
          valpha = pow2_of(vref - to);
          resc = to != vref;
          set_vref(to);
        }
#pragma unroll
        for (int r = 0; r < C::NQ; ++r) {
          const float mt = row_max(r);
          const bool need = mt > ref[r] + (kLazy + kBias);
          const float to = need ? mt - kBias : ref[r];
          alpha[r] = need ? exp2f(ref[r] - to) : 1.f;
          ref[r] = to;
          l_part[r] *= alpha[r];
          resc |= need;
        }
        if (resc && cur.j > 1) {  // O holds the group's earlier tiles of the segment: rescale it once they are done
          warp_wait(pv_done + 8 * grp, (u - 1) & 1, failed);
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < C::NB * C::NP; x += 16) {
              // 16 columns: of NQ = 16 rows one term, of fewer rows several
            float o[16];
            tmem_load<16>(o_cols + C::NP * C::NB * grp + x, o);
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] *= alpha[r % C::NQ] * valpha;
            tmem_st16(o_cols + C::NP * C::NB * grp + x, o);
          }
          tmem_st_wait();
        }
      }
      const float vs = C::KV8 ? ksvs.y * vunit[0] * vunit[1] : kUnit16;
      float w[C::NQ];
#pragma unroll
      for (int r = 0; r < C::NQ; ++r) {
        w[r] = exp2f(sc[r] - ref[r]);
        l_part[r] += w[r];
        w[r] *= vs;
      }

      // P(i) -> the group's buffer; its last reader, P.V(i - 2), must be done
      if (u >= 1) warp_wait(pv_done + 8 * grp, (u - 1) & 1, failed);
      if (tq == 0) edge[grp] = clear;
      // Column n of a position: byte or bf16 n % 16 or n % 8 of its 16 bytes in a block of columns. So a position's
      // columns leave its thread by a few 16-byte stores (a byte each: 96 stores for 16 rows).
      constexpr int kBlocks = C::PP * C::NP * C::EB / 16;
      uint32_t col[4 * kBlocks] = {};
      if constexpr (C::KV8) {
#pragma unroll
        for (int r = 0; r < C::NQ; r += 4) {
          uint16_t lo[C::PT], hi[C::PT];
          six_terms<C::PP>(make_float2(w[r], w[r + 1]), lo);
          six_terms<C::PP>(make_float2(w[r + 2], w[r + 3]), hi);
#pragma unroll
          for (int j = 0; j < C::PT; ++j)
            col[(j % C::PP * C::NP + j / C::PP * C::NQ + r) / 4] = lo[j] | (static_cast<uint32_t>(hi[j]) << 16);
        }
      } else {
#pragma unroll
        for (int r = 0; r < C::NQ; r += 2) {
          float x = w[r], y = w[r + 1];
#pragma unroll
          for (int j = 0; j < C::PT; ++j) {
            const uint16_t lo = f32_to_bf16_bits(x), hi = f32_to_bf16_bits(y);
            col[(j * C::NQ + r) / 2] = lo | (static_cast<uint32_t>(hi) << 16);
            x -= bf16_bits_to_f32(lo);
            y -= bf16_bits_to_f32(hi);
          }
        }
      }
      uint4* pbuf = reinterpret_cast<uint4*>(smem + C::OFF_P + grp * C::P_BYTES) + pl;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        pbuf[b * kTile] = make_uint4(col[4 * b], col[4 * b + 1], col[4 * b + 2], col[4 * b + 3]);
      fence_proxy_async_smem();  // P -> the tensor cores' view of shared memory
      tc_fence_before();
      mbar_arrive(p_ready + 8 * grp);

      // A position that takes no part has weight 0, but its V row may hold
      // anything, NaN too: it is cleared before the MMAs read the slot.
      if (clear) {
#pragma unroll 1
        for (int p = 0; p < C::NB; ++p) {
          const int slot = C::RK + (i * C::NB + p) % C::RV;
          warp_wait(v_here + 8 * (grp * C::NB + p), cleared & 1, failed);
          if (dead_row) {
#pragma unroll 1
            for (int x = 0; x < C::SW * C::CH; x += 16)
              *reinterpret_cast<uint4*>(smem + slot * C::SLOT + x / C::SW * C::CHUNK + pl * C::SW + x % C::SW) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          mbar_arrive(v_clean + 8 * (grp * C::NB + p));
        }
        ++cleared;
      }

      if (cur.j + 2 >= cur.n) {
        // ---- epilogue, after the group's last tile of the segment: its row sums, then this thread's
        // dim of blocks of dims. Where both groups had tiles they exchange their statistics, and each takes
        // half of the output from both accumulators. In loops: the code runs once or twice a block, so what
        // it costs is fetching it (unrolled it took 25,000 cycles).
        const bool both = cur.n > 1;
        const bool direct = cur.begins && cur.ends;
        const int slot = 2 * c + (cur.begins ? 1 : 0);
        const float lsum = rowreduce<C::NQ>(l_part, lane, AddOp());
        if (lane % kPer == 0) {
          sums[(lane / kPer) * kSoftWarps + sw] = lsum;
          if (sw == 0) refs[lane / kPer] = ref_lane;
        }
        named_bar_sync(BAR_GROUP + grp, kSoft);
        warp_wait(pv_done + 8 * grp, u & 1, failed);
        if (tq < C::NQ) {
          const float4 t4 = *reinterpret_cast<const float4*>(sums + tq * kSoftWarps);
          stat[grp * C::NQ + tq] = make_float2(refs[tq], (t4.x + t4.y) + (t4.z + t4.w));  // fixed order
          if (tq == 0) vrefs[grp] = vref;
        }
        if (both) named_bar_sync(BAR_BOTH, 2 * kSoft);
        if (tq < C::NQ) {
          float2 s0 = stat[tq], s1 = stat[C::NQ + tq];
          if (!both && grp == 0) s1 = make_float2(kNone, 0.f);
          if (!both && grp == 1) s0 = make_float2(kNone, 0.f);
          const float m = fmaxf(s0.x, s1.x);
          const float e0 = exp2f(s0.x - m), e1 = exp2f(s1.x - m);
          const float l = e0 * s0.y + e1 * s1.y;
          const float by = l == 0.f ? 0.f : 1.f / l;
          if constexpr (C::KV8) {  // times 2^vref, but for 2^-64 that the output takes where that is very small
            const int v_other = both ? vrefs[1 - grp] : vref, low = max(vref, v_other) < -64 ? -64 : 0;
            fac[tq] = e0 * by * pow2_of((grp == 0 ? vref : v_other) - low);
            fac[C::NQ + tq] = e1 * by * pow2_of((grp == 1 ? vref : v_other) - low);
            if (tq == 0) vrefs[2 + grp] = low;
          } else {
            fac[tq] = e0 * by * (1.f / kUnit16);
            fac[C::NQ + tq] = e1 * by * (1.f / kUnit16);
          }
          if (!direct && tq < G && (!both || grp == 0))
            reinterpret_cast<float2*>(a.ws_ml)[static_cast<size_t>(slot) * G + tq] = make_float2(m, l);
        }
        named_bar_sync(BAR_GROUP + grp, kSoft);
        tc_fence_after();
        const bool low = C::KV8 && vrefs[2 + grp] != 0;
        // with one block of dims the groups share its rows
        const int row0 = both && C::NB == 1 ? grp * (C::NQ / 2) : 0;
        const int row1 = min(G, both && C::NB == 1 ? row0 + C::NQ / 2 : C::NQ);
#pragma unroll 1
        for (int mb = both && C::NB > 1 ? grp : 0; mb < C::NB; mb += both && C::NB > 1 ? 2 : 1) {
          float x[C::NQ];
#pragma unroll
          for (int r = 0; r < C::NQ; ++r) x[r] = 0.f;
          // the groups' accumulators, and their terms, in fixed order, 16 columns at a time
          constexpr int kLoads = C::NP / 16, kTerms = 16 / C::NQ;
#pragma unroll 1
          for (int n = both ? 0 : grp * kLoads; n < (both ? 2 : grp + 1) * kLoads; ++n) {
            const int k = n / kLoads, part_no = n % kLoads;
            float o[16];
            tmem_load<16>(o_cols + C::NP * (C::NB * k + mb) + 16 * part_no, o);
#pragma unroll
            for (int j = 0; j < kTerms; ++j) {
              const int term = part_no * kTerms + j;
              if (term >= C::PT / C::PP) break;  // columns of no term hold anything
              const float by = C::KV8 ? __uint_as_float(static_cast<uint32_t>(127 - 4 * C::PP * term) << 23) : 1.f;
#pragma unroll
              for (int r = 0; r < C::NQ; ++r) x[r] += fac[k * C::NQ + r] * (by * o[j * C::NQ + r]);
            }
          }
          if (low) {
#pragma unroll
            for (int r = 0; r < C::NQ; ++r) x[r] *= 0x1p-64f;
          }
          const int d = mb * 128 + pl;  // O^T lanes are head dims
          if (pl < C::DB) {
            const size_t out0 = (static_cast<size_t>(cur.b) * a.NH + static_cast<size_t>(cur.kvh) * G) * C::HS + d;
            float* to32 = direct ? (a.out_f32 ? a.out_f32 + out0 : nullptr)
                                 : a.ws_o + static_cast<size_t>(slot) * G * C::HS + d;
#pragma unroll
            for (int r = 0; r < C::NQ; ++r) {
              if (r >= row0 && r < row1) {
                if (direct) a.out[out0 + r * C::HS] = f32_to_bf16_bits(x[r]);
                if (to32) to32[r * C::HS] = x[r];
              }
            }
          }
        }
        // the accumulators are free for the next segment (256 arrivals each)
        tc_fence_before();
        mbar_arrive(o_free + 8 * grp);
        mbar_arrive(o_free + 8 * (both ? 1 - grp : grp));
      }
      cur = nxt;
      page = next_page;
      ksvs = next_ksvs;
      nxt = after;
      next_page = after_page;
      i += 2;
    }
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

  // release the tensor memory once every warp is done with it
  tc_fence_before();
  __syncthreads();
  if (warp == W_QK) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
  // No copy may be in flight when the block leaves, also where a wait gave up:
  // the last phase of each slot (bounded, own flag).
  if (work && (warp == W_K || warp == W_V)) {
    const int ring = warp == W_K ? C::RK : C::RV, slot0 = warp == W_K ? 0 : C::RK;
    bool dfail = false;
    for (int k = 0; k < ring && k < slots_used; ++k)
      warp_wait(full + 8 * (slot0 + k), ((slots_used - 1 - k) / ring) & 1, dfail);
  }
}

// ------------------------------------------------------------------- the merge

constexpr int kMergeThreads = 256;

// A unit that lies in the shares c0 .. c1 left a partial in each: the mean of its values, as the output has them (in
// range whatever V's scales are), the reference and the sum of its weights. Block c in
// [c0, c1) takes its part of the unit's G * HS outputs: one item is four dims
// of a row, whose partials are summed by several threads and then in fixed
// order.
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedArgs a) {
  __shared__ float4 acc[kMergeThreads];
  extern __shared__ float factor[];  // [rows of this block][parts]
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.NH / a.NKV;
  const Cut cut = reinterpret_cast<const Cut*>(a.cuts)[c];
  if (cut.c0 < 0) return;
  const int row_items = a.HS / 4, items = G * row_items;
  const int helpers = cut.c1 - cut.c0, parts = helpers + 1;
  const int each = (items + helpers - 1) / helpers;
  const int i0 = (c - cut.c0) * each, i1 = min(items, i0 + each);
  if (i0 >= i1) return;
  const int r0 = i0 / row_items, r1 = (i1 - 1) / row_items;
  // the share c0 holds the unit's beginning, the others continue it
  auto slot_of = [&](int part) { return 2 * (cut.c0 + part) + (part == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml);
  const float4* parts_o = reinterpret_cast<const float4*>(a.ws_o);
  for (int base = i0; base < i1; base += kMergeThreads) {
    const int n = min(kMergeThreads, i1 - base);  // items of this turn
    const int groups = kMergeThreads / n;         // threads of an item
    const int item = base + tid % n, g = tid / n;
    const int r = item / row_items, d = item % row_items;
    // the first partials are on their way while the factors are made
    constexpr int kAhead = 8;
    float4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int p = g + j * groups;
      x[j] = g < groups && p < parts ? parts_o[(static_cast<size_t>(slot_of(p)) * G + r) * row_items + d]
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (base == i0) {
      for (int q = r0 + warp; q <= r1; q += kMergeThreads / 32) {
        // a lane's parts in registers, read once (more than 256 parts: the rest twice)
        constexpr int kHeld = 8;
        float2 y[kHeld];
        float m = kNegInf;  // every part has a finite reference
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          const int p = lane + 32 * j;
          y[j] = p < parts ? ml[static_cast<size_t>(slot_of(p)) * G + q] : make_float2(kNegInf, 0.f);
          m = fmaxf(m, y[j].x);
        }
        for (int p = lane + 32 * kHeld; p < parts; p += 32) m = fmaxf(m, ml[static_cast<size_t>(slot_of(p)) * G + q].x);
        for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
        // each part's share of all weights: the output is the mean of the parts' means, with these factors
        float l = 0.f;
        auto weight = [&](int p) {
          const float2 v = ml[static_cast<size_t>(slot_of(p)) * G + q];
          return exp2f(v.x - m) * v.y;
        };
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          y[j].y *= exp2f(y[j].x - m);
          l += y[j].y;
        }
        for (int p = lane + 32 * kHeld; p < parts; p += 32) l += weight(p);
        for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
        const float by = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
          if (lane + 32 * j < parts) factor[(q - r0) * parts + lane + 32 * j] = y[j].y * by;
        for (int p = lane + 32 * kHeld; p < parts; p += 32) factor[(q - r0) * parts + p] = weight(p) * by;
      }
      __syncthreads();
    }
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* f = factor + (r - r0) * parts;
    auto add = [&](const float4& y, float w) {
      s.x += w * y.x;
      s.y += w * y.y;
      s.z += w * y.z;
      s.w += w * y.w;
    };
    if (g < groups) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (g + j * groups < parts) add(x[j], f[g + j * groups]);
#pragma unroll 4
      for (int p = g + kAhead * groups; p < parts; p += groups)
        add(parts_o[(static_cast<size_t>(slot_of(p)) * G + r) * row_items + d], f[p]);
      acc[tid] = s;
    }
    __syncthreads();
    if (g == 0) {
#pragma unroll 4
      for (int j = 1; j < min(groups, parts); ++j) add(acc[j * n + tid], 1.f);
      const size_t at = (static_cast<size_t>(cut.b) * a.NH + static_cast<size_t>(cut.kvh) * G + r) * a.HS + 4 * d;
      const uint32_t lo = f32_to_bf16_bits(s.x) | (static_cast<uint32_t>(f32_to_bf16_bits(s.y)) << 16);
      const uint32_t hi = f32_to_bf16_bits(s.z) | (static_cast<uint32_t>(f32_to_bf16_bits(s.w)) << 16);
      *reinterpret_cast<uint2*>(a.out + at) = make_uint2(lo, hi);
      if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + at) = s;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ the launch

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
  // the rows that a softmax thread works on: 4, 8 or 16, as the group has
  const int G = a.NH / a.NKV;
  if (G <= 4) return launch_cfg<Cfg<HS, KV8, 4>>(a, stream);
  if (G <= 8) return launch_cfg<Cfg<HS, KV8, 8>>(a, stream);
  return launch_cfg<Cfg<HS, KV8, 16>>(a, stream);
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
