/*
 * fd_paged_attn.h - C ABI of libfd.so for a KV cache kept in pages: single-token
 * attention over it, the writer of new tokens, and the bookkeeping of its
 * pages (growing, forking, freeing, compacting, copying). Status codes,
 * streams, alignment and the device error word are those of fd_decode_attn.h.
 *
 * The cache of one layer is a pool of pages of page_size tokens each:
 *     k_pages, v_pages  [num_pages][NKV][page_size][HS]  bf16 (FD_KV_BF16) or
 *                       E4M3 codes (FD_KV_E4M3)
 *     k_scale, v_scale  fp32 [num_pages][NKV], FD_KV_E4M3 only: a block of
 *                       page_size tokens of one head has one scale for K and
 *                       one for V, value = E4M3(code) * scale; scales are >= 0
 * Every layer's pool uses the same bookkeeping:
 *     table  int32 [B][max_pages]  page of positions [j * page_size,
 *                                  (j + 1) * page_size) of sequence b; -1: none
 *     lens   int32 [B]             tokens of sequence b
 *     refs   int32 [num_pages]     how many rows hold the page; 0: free
 * Position p of sequence b is slot p % page_size of page table[b][p / page_size].
 *
 * One decode step:
 *     fd_pages_reserve   room for the step's tokens; raises lens; lists the
 *                        shared last pages that have to be copied
 *     fd_pages_copy      copies them, in every layer (an empty list is cheap)
 *     then in each layer fd_paged_append (K and V of the new tokens) and
 *     fd_paged_attn (lens counts the new token, as for fd_decode_attn).
 * Everything is read on the device, nothing synchronises the host, so the
 * whole step can be captured in a CUDA graph.
 *
 * Conventions beside those of fd_decode_attn.h:
 *   - page_size is 16, 32, 64 or 128; HS is 64, 128, 256 or 512;
 *     max_pages * page_size is at most 2^31 - 4097, and for fd_paged_attn and
 *     fd_paged_append B * (max_pages * page_size / 32 + 32) is below 2^31: close
 *     to 2^36 positions in all (else FD_ERR_UNSUPPORTED).
 *   - Tensors are densely packed but for k_new and v_new of fd_paged_append,
 *     whose rows (tokens) may be any multiple of 8 elements apart.
 *   - q, out, the pages, k_new, v_new and workspaces are 16-byte aligned; the
 *     int32 and fp32 arrays 4-byte aligned (else FD_ERR_ALIGNMENT).
 *   - Two calls that overlap on the GPU must not share a workspace, nor may one
 *     of them write what the other uses.
 */
#ifndef FD_PAGED_ATTN_H_
#define FD_PAGED_ATTN_H_

#include "fd_decode_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device error word (fd_get_device_error). */
enum {
  FD_DEVERR_PAGE_ID = 1u << 4,        /* a needed table entry names no page of the pool, or a list names
                                         a row or a page that is not there; it was left out */
  FD_DEVERR_PAGES_EXHAUSTED = 1u << 5 /* fd_pages_reserve: some sequence got no pages (its granted is 0) */
};

/*
 * Plan of fd_paged_attn_ex. The work is the stream of every (sequence, KV
 * head)'s live band in pieces of `granule` positions, each band counted as
 * `min_share` pieces more than it has, and dealt to
 * `blocks` thread blocks in equal consecutive shares on the device (the
 * lengths are read there): a block may end one band and begin the next. A band
 * that lies in several shares leaves one partial in each, which a
 * second kernel merges.
 */
typedef struct {
  int blocks;             /* thread blocks of the attention kernel (persistent) */
  int granule;            /* positions: shares begin at multiples of it in a band */
  int min_share;          /* a block's share is at least this many granules, and a band counts as that many more */
  int num_sms;            /* SM count the plan assumed */
  int kv_dtype;           /* FD_KV_BF16 or FD_KV_E4M3 */
  size_t workspace_bytes; /* bytes of workspace fd_paged_attn_ex needs; no byte of it needs a value */
  int B, NH, NKV, HS, page_size, max_pages, window; /* the shape the plan was made for */
} fd_paged_plan_t;

/*
 * fd_paged_plan: plan for the given shape on CUDA device `device`; a pure host
 * computation plus device attribute queries. fd_paged_plan_sms: the same for a
 * GPU of num_sms (at most 1024) SMs, without touching a device.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_UNSUPPORTED, FD_ERR_CUDA.
 */
int fd_paged_plan(int B, int NH, int NKV, int HS, int page_size, int max_pages, int window, int device,
                  int kv_dtype, fd_paged_plan_t* plan);
int fd_paged_plan_sms(int B, int NH, int NKV, int HS, int page_size, int max_pages, int window, int num_sms,
                      int kv_dtype, fd_paged_plan_t* plan);

/*
 * fd_paged_attn: one query token per sequence over the paged cache. With
 * kvh = h / (NH / NKV) and band_b = [max(0, len_b - window), len_b) (window <= 0:
 * [0, len_b)), for every sequence b and query head h
 *     s_p    = scale * dot(q[b][h], K_p),  p in band_b
 *     out[b][h] = sum_p softmax(s)_p * V_p
 * where K_p, V_p are the values at position p of head kvh. q and out are bf16
 * [B][NH][HS], lens int32 [B]. scale <= 0 selects 1/sqrt(HS). A sequence of
 * length 0 gives a zero row. Only slots of the live band take part: what the
 * other slots of a page hold (NaN, say) has no effect, and pages outside the
 * band are not read, so their table entries may be -1. An infinity in a live V
 * gives NaN (the terms below add it times 0). A row of which no score is above
 * -infinity is zero.
 * An entry that names no page raises FD_DEVERR_PAGE_ID and its positions are
 * left out; len_b < 0 counts as 0 (FD_DEVERR_LEN_NEGATIVE); len_b above
 * max_pages * page_size counts as that (FD_DEVERR_LEN_CLAMPED).
 * Arithmetic, E4M3: q is split into three E4M3 terms (exact for elements within
 * 2^17 of the row's largest, else off by 2^-25 of that; HS 512 with NH / NKV > 8:
 * two terms, 2^13 and 2^-21) and the softmax
 * weights, times their block's V scale, into six (off by 2^-24 of themselves or
 * 2^-32 of the largest weight times the largest scale; HS 512 with NH / NKV > 8:
 * 2^-30 of that, so n positions of weights that are that small may add n times
 * as much to the error); products accumulate in fp32. Every scale that is not
 * negative is taken, 0 and subnormals too. bf16: q enters as it
 * is, the weights, at most 1, as three bf16 terms (2^-24); like the products of
 * any softmax in fp32, theirs with V overflow where they add up to 2^128.
 * fd_paged_attn makes its plan for the current device and uses a workspace
 * the library owns, one per (device, stream; the per-thread default stream is a
 * stream of its own in each thread): the first call for a pair
 * allocates it (not while the stream is captured: FD_ERR_WORKSPACE), large
 * enough for every shape, and it is kept until fd_release, so graphs captured
 * on one stream share it and must not be replayed at the same time.
 * fd_paged_attn_ex takes a plan, a workspace of
 * plan->workspace_bytes and an optional fp32 copy of the output, and allocates
 * nothing. Shapes: NH % NKV == 0, NH / NKV <= 16; B, NKV <= 65535; B == 0 is a
 * no-op.
 * Errors: every FD_ERR_* code but FD_ERR_SCRATCH_LIMIT.
 */
int fd_paged_attn(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                  const float* v_scale, void* out, const int* table, const int* lens, int B, int NH, int NKV,
                  int HS, int page_size, int num_pages, int max_pages, int window, float scale, int kv_dtype,
                  fd_stream_t stream);
int fd_paged_attn_ex(const fd_paged_plan_t* plan, void* workspace, size_t workspace_bytes, float* out_f32,
                     const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                     const float* v_scale, void* out, const int* table, const int* lens, int B, int NH, int NKV,
                     int HS, int page_size, int num_pages, int max_pages, int window, float scale,
                     fd_stream_t stream);

/*
 * fd_paged_append: write K and V of new tokens into the pages. Sequence b's new
 * tokens are rows [start[b], start[b] + n_b) of k_new and v_new (bf16 [T][NKV][HS],
 * rows k_stride and v_stride elements apart), with n_b = start[b + 1] - start[b],
 * and go to positions [lens[b] - n_b, lens[b]): lens counts them already, and
 * the table has their pages (fd_pages_reserve does both). start is int32
 * [B + 1], rising from 0 to at most T; start == NULL is one token for each
 * sequence (T == B). count (int32 [B], may be NULL) takes tokens away: n_b
 * becomes min(n_b, count[b]), at least 0 - with fd_pages_reserve's `granted`
 * a sequence that got no room writes nothing. Rows behind a sequence's n_b are
 * not read. A page that is written must be in no other row of the table.
 * FD_KV_E4M3: for each page and head that gets tokens, with a the largest
 * finite |x| among them,
 *     s = max(old scale if the page holds earlier tokens of the sequence, s_a),
 *     s_a = least power of two with a <= 448 s_a, at least 2^-126 (0 if a = 0),
 *     code(x) = nearest E4M3 value of x / s, ties to even; NaN where x is not
 *     finite; 0 where s = 0,
 * and where s rises over the old scale the page's earlier codes become
 * nearest(code * (old scale / s)): exact for scales that are powers of two, but for
 * values that fall below E4M3's smallest. Slots behind the last token are left
 * as they were. A page's scale is taken as new when its slot 0 is written.
 * A needed table entry that names no page raises FD_DEVERR_PAGE_ID and its
 * tokens are left out; so are tokens at positions from max_pages * page_size
 * on and rows outside [0, T). A token whose position would be negative (the one
 * of a sequence of length 0) is left out and raises nothing. With T == 0 nothing
 * is done, and max_pages may be 0.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_UNSUPPORTED, FD_ERR_ALIGNMENT, FD_ERR_CUDA.
 */
int fd_paged_append(const void* k_new, const void* v_new, void* k_pages, void* v_pages, float* k_scale,
                    float* v_scale, const int* table, const int* lens, const int* start, const int* count, int B,
                    int T, int NKV, int HS, int page_size, int num_pages, int max_pages, long long k_stride,
                    long long v_stride, int kv_dtype, fd_stream_t stream);

/*
 * fd_pages_workspace_bytes: workspace of fd_pages_reserve and
 * fd_pages_compact: 4 * (num_pages + 4 * B + 256). No byte of it needs a value.
 */
size_t fd_pages_workspace_bytes(int B, int num_pages);

/*
 * A list of moves: int32 [2 * (room + 1)]. moves[0] is the number of moves n,
 * moves[1] the number of free pages that were not handed out (a page that this
 * call of fd_pages_reserve took from its last owner is free beside them),
 * moves[2 + 2 i] and moves[3 + 2 i] the source and the destination of move
 * i < n; entries behind them are left as they were.
 *
 * fd_pages_reserve: room for grow[b] more tokens (int32 [B]; NULL: one for
 * each; <= 0: none) of every sequence. A sequence needs a page for each
 * page_size positions it enters, and one more where its last page is begun and
 * held by other rows too (refs > 1): that page is replaced in its row by a new
 * one, listed as a move, and loses the row as an owner - also where every owner
 * does so in one call. Free pages are handed out in rising order, sequences
 * served in order, a sequence's replaced page first; a sequence is granted its
 * tokens when the pages needed by it and by all before it are free, or when it
 * needs none, and when its row is long enough. granted[b] (int32 [B]) is
 * grow[b] or 0, and lens[b] rises by it. Where 0 was granted for more, the row
 * stays as it was and FD_DEVERR_PAGES_EXHAUSTED is raised (FD_DEVERR_PAGE_ID
 * where its last page's entry names no page, which also denies it).
 * moves needs room for B.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_UNSUPPORTED, FD_ERR_ALIGNMENT,
 * FD_ERR_WORKSPACE, FD_ERR_CUDA.
 */
int fd_pages_reserve(int* table, int* lens, int* refs, const int* grow, int* granted, int* moves, void* workspace,
                     size_t workspace_bytes, int B, int max_pages, int num_pages, int page_size,
                     fd_stream_t stream);

/*
 * fd_pages_fork: new rows from old ones: table_out[i] = table[parent[i]],
 * lens_out[i] = lens[parent[i]] for i < B_out; parent[i] = -1 gives an empty row
 * (all -1, length 0), any other value outside [0, B) too, with FD_DEVERR_PAGE_ID.
 * refs loses the old rows as owners and gains the new ones: a parent named twice
 * is forked, one not named is freed, and its pages that nobody else holds are
 * free. table_out and lens_out must not overlap table and lens.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_ALIGNMENT, FD_ERR_CUDA.
 */
int fd_pages_fork(const int* table, const int* lens, const int* parent, int* table_out, int* lens_out, int* refs,
                  int B, int B_out, int max_pages, int num_pages, fd_stream_t stream);

/*
 * fd_pages_free: lens[b] becomes min(lens[b], keep[b]) (int32 [B]; NULL: every
 * token is kept; < 0 counts as 0), and the row gives up its pages behind that length.
 * With window > 0 it also gives up the pages that hold no position of
 * [max(0, lens[b] - window), lens[b]): what sliding-window layers no longer
 * read. Given-up entries become -1 and their pages lose the row as an owner.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_UNSUPPORTED, FD_ERR_ALIGNMENT, FD_ERR_CUDA.
 */
int fd_pages_free(int* table, int* lens, int* refs, const int* keep, int window, int B, int max_pages,
                  int num_pages, int page_size, fd_stream_t stream);

/*
 * fd_pages_compact: move the pages in use together: with n pages in use
 * (refs > 0), the i-th page in use with a number >= n takes the i-th free
 * number < n. refs follows, the table names the new numbers, and the moves are
 * listed for fd_pages_copy; no page is both a source and a destination.
 * Afterwards pages [n, num_pages) are free. moves needs room for
 * num_pages / 2.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_ALIGNMENT, FD_ERR_WORKSPACE, FD_ERR_CUDA.
 */
int fd_pages_compact(int* table, int* refs, int* moves, void* workspace, size_t workspace_bytes, int B,
                     int max_pages, int num_pages, fd_stream_t stream);

/*
 * fd_pages_copy: copy the listed pages, K, V and (FD_KV_E4M3) their scales, in
 * each of `layers` pools that lie one behind the other: k_pages and v_pages
 * [layers][num_pages][NKV][page_size][HS], scales [layers][num_pages][NKV]. The
 * number of moves is read on the device; `room` is the room of the list, and
 * no more moves than that are made. A move that names no page is left out
 * (FD_DEVERR_PAGE_ID). A page must not be the destination of two moves, nor a
 * source and a destination.
 * Errors: FD_ERR_INVALID_ARG, FD_ERR_UNSUPPORTED, FD_ERR_ALIGNMENT, FD_ERR_CUDA.
 */
int fd_pages_copy(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int* moves, int room,
                  int layers, int num_pages, int NKV, int page_size, int HS, int kv_dtype, fd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FD_PAGED_ATTN_H_ */
