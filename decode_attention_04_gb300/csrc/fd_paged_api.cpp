// Host side of the paged cache: argument checks, the plan, the library-owned
// workspace, and the exported C entry points declared in fd_paged_attn.h.

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>

#include <cuda_runtime.h>

#include "fd_paged.h"
#include "fd_paged_attn.h"

namespace {

constexpr int kMaxGroup = 16;
constexpr int kMaxHS = 512;
constexpr int kMaxPositions = INT_MAX - 4096;  // positions are int32, and a tile may reach past the last

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool supported_hs(int HS) { return HS == 64 || HS == 128 || HS == 256 || HS == 512; }
bool supported_page(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }
bool valid_dtype(int t) { return t == FD_KV_BF16 || t == FD_KV_E4M3; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int check_shape(int B, int NH, int NKV, int HS, int page_size, int max_pages, int kv_dtype) {
  if (B < 0 || NH <= 0 || NKV <= 0 || max_pages <= 0 || !valid_dtype(kv_dtype)) return FD_ERR_INVALID_ARG;
  if (B > 65535 || NKV > 65535) return FD_ERR_INVALID_ARG;
  if (!supported_hs(HS) || !supported_page(page_size)) return FD_ERR_UNSUPPORTED;
  if (NH % NKV != 0 || NH / NKV > kMaxGroup) return FD_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > kMaxPositions) return FD_ERR_UNSUPPORTED;  // lens are int32
  // the kernels count the 32-position granules of one head, and 64 KB of them more for each sequence, in 32 bits
  if (static_cast<long long>(B) * (static_cast<long long>(max_pages) * page_size / 32 + 32) > INT_MAX)
    return FD_ERR_UNSUPPORTED;
  return FD_OK;
}

// Partials: one per share's first and last band, G rows of HS floats; then
// their (m, l); then 16 bytes a share on the unit that its end cuts.
size_t ws_o_bytes(int blocks, int G, int HS) {
  return round_up(static_cast<size_t>(2) * blocks * G * HS * sizeof(float), 256);
}
size_t ws_ml_bytes(int blocks, int G) { return round_up(static_cast<size_t>(2) * blocks * G * 2 * sizeof(float), 256); }
size_t ws_bytes(int blocks, int G, int HS) {
  return ws_o_bytes(blocks, G, HS) + ws_ml_bytes(blocks, G) + round_up(static_cast<size_t>(blocks) * 16, 256);
}

int make_plan(int B, int NH, int NKV, int HS, int page_size, int max_pages, int window, int num_sms, int kv_dtype,
              fd_paged_plan_t* plan) {
  if (!plan) return FD_ERR_INVALID_ARG;
  const int rc = check_shape(B, NH, NKV, HS, page_size, max_pages, kv_dtype);
  if (rc != FD_OK) return rc;
  if (num_sms <= 0 || num_sms > 1024) return FD_ERR_INVALID_ARG;  // the merge keeps 2 factors a block in shared memory
  fd_paged_plan_t p{};
  p.blocks = num_sms;
  p.granule = 32;
  // At least 64 KB of K and V a share: below that a merge of its partial costs
  // more than the SMs left idle (256 positions of 8 heads of 128, E4M3, in
  // shares of 8 KB 9.8 us, of 32 KB 9.2, of 64 KB, whole bands, 7.6; 1024
  // positions of 8 heads of 256 in 32 KB 10.9, 64 KB 10.5, 128 KB 11.1).
  p.min_share = std::max(1, (64 << 10) / (2 * p.granule * HS * (kv_dtype == FD_KV_E4M3 ? 1 : 2)));
  p.num_sms = num_sms;
  p.kv_dtype = kv_dtype;
  p.workspace_bytes = ws_bytes(p.blocks, NH / NKV, HS);
  p.B = B;
  p.NH = NH;
  p.NKV = NKV;
  p.HS = HS;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.window = window;
  *plan = p;
  return FD_OK;
}

std::mutex g_mu;
std::map<int, int> g_sms;
std::map<std::tuple<int, uintptr_t, unsigned long long>, void*> g_ws;  // device, stream, its id where the handle is shared

int run(const fd_paged_plan_t& p, void* workspace, size_t workspace_bytes, float* out_f32, const void* q,
        const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale, void* out,
        const int* table, const int* lens, int num_pages, float scale, cudaStream_t stream) {
  if (p.B == 0) return FD_OK;
  if (!workspace || workspace_bytes < p.workspace_bytes) return FD_ERR_WORKSPACE;
  const bool kv8 = p.kv_dtype == FD_KV_E4M3;
  if (!aligned(workspace, 16) || !aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(out, 16) || (out_f32 && !aligned(out_f32, 16)) || !aligned(table, 4) || !aligned(lens, 4) ||
      (kv8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return FD_ERR_ALIGNMENT;
  if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(p.HS));
  const int G = p.NH / p.NKV;
  fd::PagedArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = k_pages;
  a.v = v_pages;
  a.k_scale = kv8 ? k_scale : nullptr;
  a.v_scale = kv8 ? v_scale : nullptr;
  a.out = static_cast<uint16_t*>(out);
  a.out_f32 = out_f32;
  a.table = table;
  a.lens = lens;
  a.ws_o = static_cast<float*>(workspace);
  a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws_o_bytes(p.blocks, G, p.HS));
  a.cuts = reinterpret_cast<char*>(a.ws_ml) + ws_ml_bytes(p.blocks, G);
  a.B = p.B;
  a.NH = p.NH;
  a.NKV = p.NKV;
  a.HS = p.HS;
  a.P = p.page_size;
  a.num_pages = num_pages;
  a.max_pages = p.max_pages;
  a.window = p.window;
  a.blocks = p.blocks;
  a.min_share = p.min_share;
  a.kv8 = kv8;
  a.withhold_tile = fd::debug_withhold_tile();
  a.scale_log2 = scale * 1.4426950408889634f;
  return fd::launch_paged_attn(a, stream) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

int check_call(const void* q, const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale,
               const void* out, const int* table, const int* lens, int num_pages, int kv_dtype) {
  if (num_pages <= 0) return FD_ERR_INVALID_ARG;
  if (!q || !k_pages || !v_pages || !out || !table || !lens) return FD_ERR_INVALID_ARG;
  if (kv_dtype == FD_KV_E4M3 && (!k_scale || !v_scale)) return FD_ERR_INVALID_ARG;
  return FD_OK;
}

// Arrays of the bookkeeping: sizes and the 4-byte alignment of each.
int check_book(int B, int max_pages, int num_pages) {
  if (B < 0 || B > 65535 || max_pages <= 0 || num_pages <= 0) return FD_ERR_INVALID_ARG;
  if (num_pages > INT_MAX - 4 * 65536 - 1024) return FD_ERR_INVALID_ARG;
  return FD_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

int status(cudaError_t e) { return e == cudaSuccess ? FD_OK : FD_ERR_CUDA; }

int current_sms(int* sms) {
  int device = 0;
  return cudaGetDevice(&device) == cudaSuccess ? fd::device_sm_count(device, sms) : FD_ERR_CUDA;
}

}  // namespace

namespace fd {

int device_sm_count(int device, int* sms) try {
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_sms.find(device);
  if (it != g_sms.end()) {
    *sms = it->second;
    return FD_OK;
  }
  int v = 0;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || v <= 0) return FD_ERR_CUDA;
  g_sms[device] = v;
  *sms = v;
  return FD_OK;
} catch (...) {  // the map's memory: no exception leaves a C entry
  return FD_ERR_CUDA;
}

// One buffer per (device, stream), large enough for every shape on that device, so
// it never grows and a captured graph's pointer stays good until fd_release.
// The handle of the per-thread default stream names another stream in each thread.
int paged_workspace(int device, cudaStream_t stream, size_t bytes, void** ptr) try {
  unsigned long long id = 0;
  if (stream == cudaStreamPerThread && cudaStreamGetId(stream, &id) != cudaSuccess) return FD_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  void*& w = g_ws[{device, reinterpret_cast<uintptr_t>(stream), id}];
  if (!w) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return FD_ERR_CUDA;
    if (cap != cudaStreamCaptureStatusNone) return FD_ERR_WORKSPACE;
    if (cudaMalloc(&w, bytes) != cudaSuccess) {
      w = nullptr;
      return FD_ERR_CUDA;
    }
  }
  *ptr = w;
  return FD_OK;
} catch (...) {
  return FD_ERR_CUDA;
}

void paged_release() {
  std::lock_guard<std::mutex> lk(g_mu);
  for (auto& kv : g_ws) {
    if (!kv.second) continue;
    int prev = 0;
    cudaGetDevice(&prev);
    cudaSetDevice(std::get<0>(kv.first));
    cudaFree(kv.second);
    cudaSetDevice(prev);
  }
  g_ws.clear();
}

}  // namespace fd

extern "C" {

int fd_paged_plan_sms(int B, int NH, int NKV, int HS, int page_size, int max_pages, int window, int num_sms,
                      int kv_dtype, fd_paged_plan_t* plan) {
  return make_plan(B, NH, NKV, HS, page_size, max_pages, window, num_sms, kv_dtype, plan);
}

int fd_paged_plan(int B, int NH, int NKV, int HS, int page_size, int max_pages, int window, int device, int kv_dtype,
                  fd_paged_plan_t* plan) {
  if (!plan) return FD_ERR_INVALID_ARG;
  int rc = check_shape(B, NH, NKV, HS, page_size, max_pages, kv_dtype);
  if (rc != FD_OK) return rc;
  int sms = 0;
  rc = fd::device_sm_count(device, &sms);
  if (rc != FD_OK) return rc;
  return make_plan(B, NH, NKV, HS, page_size, max_pages, window, sms, kv_dtype, plan);
}

int fd_paged_attn_ex(const fd_paged_plan_t* plan, void* workspace, size_t workspace_bytes, float* out_f32,
                     const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                     const float* v_scale, void* out, const int* table, const int* lens, int B, int NH, int NKV,
                     int HS, int page_size, int num_pages, int max_pages, int window, float scale,
                     fd_stream_t stream) {
  if (!plan) return FD_ERR_INVALID_ARG;
  // The plan must be one that fd_paged_plan_sms gives for these sizes.
  fd_paged_plan_t want;
  int rc = make_plan(B, NH, NKV, HS, page_size, max_pages, window, plan->num_sms, plan->kv_dtype, &want);
  if (rc != FD_OK) return rc;
  if (plan->B != B || plan->NH != NH || plan->NKV != NKV || plan->HS != HS || plan->page_size != page_size ||
      plan->max_pages != max_pages || plan->window != window || plan->blocks != want.blocks ||
      plan->granule != want.granule || plan->min_share != want.min_share ||
      plan->workspace_bytes != want.workspace_bytes)
    return FD_ERR_INVALID_ARG;
  if (B == 0) return FD_OK;
  rc = check_call(q, k_pages, v_pages, k_scale, v_scale, out, table, lens, num_pages, plan->kv_dtype);
  if (rc != FD_OK) return rc;
  return run(*plan, workspace, workspace_bytes, out_f32, q, k_pages, v_pages, k_scale, v_scale, out, table, lens,
             num_pages, scale, reinterpret_cast<cudaStream_t>(stream));
}

int fd_paged_attn(const void* q, const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale,
                  void* out, const int* table, const int* lens, int B, int NH, int NKV, int HS, int page_size,
                  int num_pages, int max_pages, int window, float scale, int kv_dtype, fd_stream_t stream) {
  int rc = check_shape(B, NH, NKV, HS, page_size, max_pages, kv_dtype);
  if (rc != FD_OK) return rc;
  if (B == 0) return FD_OK;
  rc = check_call(q, k_pages, v_pages, k_scale, v_scale, out, table, lens, num_pages, kv_dtype);
  if (rc != FD_OK) return rc;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return FD_ERR_CUDA;
  fd_paged_plan_t plan;
  rc = fd_paged_plan(B, NH, NKV, HS, page_size, max_pages, window, device, kv_dtype, &plan);
  if (rc != FD_OK) return rc;
  void* ws = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rc = fd::paged_workspace(device, s, ws_bytes(plan.blocks, kMaxGroup, kMaxHS), &ws);
  if (rc != FD_OK) return rc;
  return run(plan, ws, plan.workspace_bytes, nullptr, q, k_pages, v_pages, k_scale, v_scale, out, table, lens,
             num_pages, scale, s);
}

int fd_paged_append(const void* k_new, const void* v_new, void* k_pages, void* v_pages, float* k_scale,
                    float* v_scale, const int* table, const int* lens, const int* start, const int* count, int B,
                    int T, int NKV, int HS, int page_size, int num_pages, int max_pages, long long k_stride,
                    long long v_stride, int kv_dtype, fd_stream_t stream) {
  // a batch of empty sequences has a table of no columns, and no token to write into it
  const int rc = check_shape(B, NKV, NKV, HS, page_size, T == 0 && max_pages == 0 ? 1 : max_pages, kv_dtype);
  if (rc != FD_OK) return rc;
  if (T < 0 || num_pages <= 0 || (!start && T != B)) return FD_ERR_INVALID_ARG;
  const long long row = static_cast<long long>(NKV) * HS;
  if (k_stride < row || v_stride < row) return FD_ERR_INVALID_ARG;
  if (k_stride % 8 != 0 || v_stride % 8 != 0) return FD_ERR_ALIGNMENT;
  if (B == 0 || T == 0) return FD_OK;
  const bool kv8 = kv_dtype == FD_KV_E4M3;
  if (!k_new || !v_new || !k_pages || !v_pages || !table || !lens || (kv8 && (!k_scale || !v_scale)))
    return FD_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(start, 4) || !aligned(count, 4) ||
      (kv8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return FD_ERR_ALIGNMENT;
  fd::AppendArgs a{};
  a.x[0] = static_cast<const uint16_t*>(k_new);
  a.x[1] = static_cast<const uint16_t*>(v_new);
  a.pages[0] = k_pages;
  a.pages[1] = v_pages;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.table = table;
  a.lens = lens;
  a.start = start;
  a.count = count;
  a.B = B;
  a.T = T;
  a.NKV = NKV;
  a.HS = HS;
  a.P = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.kv8 = kv8;
  return status(fd::launch_paged_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fd_pages_workspace_bytes(int B, int num_pages) {
  if (B < 0 || num_pages < 0) return 0;
  return sizeof(int) * (static_cast<size_t>(num_pages) + 4 * static_cast<size_t>(B) + fd::kPagesHeader);
}

int fd_pages_reserve(int* table, int* lens, int* refs, const int* grow, int* granted, int* moves, void* workspace,
                     size_t workspace_bytes, int B, int max_pages, int num_pages, int page_size,
                     fd_stream_t stream) {
  const int rc = check_book(B, max_pages, num_pages);
  if (rc != FD_OK) return rc;
  if (!supported_page(page_size) || static_cast<long long>(max_pages) * page_size > kMaxPositions) return FD_ERR_UNSUPPORTED;
  if (!refs || !moves || (B > 0 && (!table || !lens || !granted))) return FD_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < fd_pages_workspace_bytes(B, num_pages)) return FD_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(refs, 4) || !aligned(grow, 4) ||
      !aligned(granted, 4) || !aligned(moves, 4))
    return FD_ERR_ALIGNMENT;
  return status(fd::launch_pages_reserve(table, lens, refs, grow, granted, moves, static_cast<int*>(workspace), B,
                                         max_pages, num_pages, page_size, reinterpret_cast<cudaStream_t>(stream)));
}

int fd_pages_fork(const int* table, const int* lens, const int* parent, int* table_out, int* lens_out, int* refs,
                  int B, int B_out, int max_pages, int num_pages, fd_stream_t stream) {
  int rc = check_book(B, max_pages, num_pages);
  if (rc == FD_OK) rc = check_book(B_out, max_pages, num_pages);
  if (rc != FD_OK) return rc;
  if (!refs || (B > 0 && (!table || !lens)) || (B_out > 0 && (!parent || !table_out || !lens_out)))
    return FD_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(parent, 4) || !aligned(table_out, 4) ||
      !aligned(lens_out, 4) || !aligned(refs, 4))
    return FD_ERR_ALIGNMENT;
  const size_t row = sizeof(int) * static_cast<size_t>(max_pages);
  if (B > 0 && B_out > 0 && (overlap(table, row * B, table_out, row * B_out) || overlap(lens, 4ul * B, lens_out, 4ul * B_out)))
    return FD_ERR_INVALID_ARG;
  if (B == 0 && B_out == 0) return FD_OK;
  return status(fd::launch_pages_fork(table, lens, parent, table_out, lens_out, refs, B, B_out, max_pages, num_pages,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int fd_pages_free(int* table, int* lens, int* refs, const int* keep, int window, int B, int max_pages, int num_pages,
                  int page_size, fd_stream_t stream) {
  const int rc = check_book(B, max_pages, num_pages);
  if (rc != FD_OK) return rc;
  if (!supported_page(page_size) || static_cast<long long>(max_pages) * page_size > kMaxPositions) return FD_ERR_UNSUPPORTED;
  if (B == 0) return FD_OK;
  if (!table || !lens || !refs) return FD_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(refs, 4) || !aligned(keep, 4)) return FD_ERR_ALIGNMENT;
  return status(fd::launch_pages_free(table, lens, refs, keep, window, B, max_pages, num_pages, page_size,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int fd_pages_compact(int* table, int* refs, int* moves, void* workspace, size_t workspace_bytes, int B, int max_pages,
                     int num_pages, fd_stream_t stream) {
  int rc = check_book(B, max_pages, num_pages);
  if (rc != FD_OK) return rc;
  if (!refs || !moves || (B > 0 && !table)) return FD_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < fd_pages_workspace_bytes(B, num_pages)) return FD_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(table, 4) || !aligned(refs, 4) || !aligned(moves, 4)) return FD_ERR_ALIGNMENT;
  int sms = 0;
  rc = current_sms(&sms);
  if (rc != FD_OK) return rc;
  return status(fd::launch_pages_compact(table, refs, moves, static_cast<int*>(workspace), B, max_pages, num_pages, sms,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int fd_pages_copy(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int* moves, int room, int layers,
                  int num_pages, int NKV, int page_size, int HS, int kv_dtype, fd_stream_t stream) {
  if (room < 0 || layers < 0 || num_pages <= 0 || NKV <= 0 || NKV > 65535 || !valid_dtype(kv_dtype))
    return FD_ERR_INVALID_ARG;
  if (!supported_hs(HS) || !supported_page(page_size)) return FD_ERR_UNSUPPORTED;
  if (room == 0 || layers == 0) return FD_OK;
  const bool kv8 = kv_dtype == FD_KV_E4M3;
  if (!k_pages || !v_pages || !moves || (kv8 && (!k_scale || !v_scale))) return FD_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(moves, 4) ||
      (kv8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return FD_ERR_ALIGNMENT;
  const size_t page_bytes = static_cast<size_t>(NKV) * page_size * HS * (kv8 ? 1 : 2);
  int sms = 0;
  const int rc = current_sms(&sms);
  if (rc != FD_OK) return rc;
  return status(fd::launch_pages_copy(k_pages, v_pages, kv8 ? k_scale : nullptr, kv8 ? v_scale : nullptr, moves, room,
                                      layers, num_pages, NKV, page_bytes, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
