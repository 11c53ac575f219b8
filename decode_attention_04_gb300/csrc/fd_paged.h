// Internal interface between the host API of the paged cache (fd_paged_api.cpp)
// and its kernels (fd_paged_attn.cu, fd_pages.cu). The public interface is
// include/fd_paged_attn.h.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace fd {

struct PagedArgs {
  const uint16_t* q;       // bf16 [B][NH][HS]
  const void* k;           // [num_pages][NKV][P][HS], bf16 or E4M3
  const void* v;
  const float* k_scale;    // fp32 [num_pages][NKV] (E4M3 only)
  const float* v_scale;
  uint16_t* out;           // bf16 [B][NH][HS]
  float* out_f32;          // fp32 [B][NH][HS] or nullptr
  const int* table;        // [B][max_pages]
  const int* lens;         // [B]
  float* ws_o;             // fp32 [2 * blocks][G][HS]
  float* ws_ml;            // fp32 [2 * blocks][G][2]
  void* cuts;              // [blocks]: the unit that each share's end cuts
  int B, NH, NKV, HS, P, num_pages, max_pages, window;
  int blocks, min_share;
  int kv8;
  int withhold_tile;       // test hook: a block's copy warps stop at this tile of theirs (a huge value: off)
  float scale_log2;        // scale * log2(e)
};

struct AppendArgs {
  const uint16_t* x[2];    // k_new, v_new: bf16 rows
  void* pages[2];
  float* scale[2];
  long long stride[2];     // elements between rows
  const int* table;
  const int* lens;
  const int* start;        // [B + 1] or nullptr: one token each
  const int* count;        // [B] or nullptr
  int B, T, NKV, HS, P, num_pages, max_pages;
  int kv8;
};

constexpr int kPagesHeader = 256;  // ints at the head of the bookkeeping workspace

cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_pages_reserve(int* table, int* lens, int* refs, const int* grow, int* granted, int* moves, int* ws,
                                 int B, int max_pages, int num_pages, int P, cudaStream_t stream);
cudaError_t launch_pages_fork(const int* table, const int* lens, const int* parent, int* table_out, int* lens_out,
                              int* refs, int B, int B_out, int max_pages, int num_pages, cudaStream_t stream);
cudaError_t launch_pages_free(int* table, int* lens, int* refs, const int* keep, int window, int B, int max_pages,
                              int num_pages, int P, cudaStream_t stream);
cudaError_t launch_pages_compact(int* table, int* refs, int* moves, int* ws, int B, int max_pages, int num_pages,
                                 int sms, cudaStream_t stream);
cudaError_t launch_pages_copy(void* k, void* v, float* ks, float* vs, const int* moves, int room, int layers,
                              int num_pages, int NKV, size_t page_bytes, int sms, cudaStream_t stream);

// The device error words of the paged units (OR into *err, then clear).
cudaError_t read_and_clear_device_error_paged(unsigned int* err);
cudaError_t read_and_clear_device_error_pages(unsigned int* err);
cudaError_t set_wait_limit_paged(unsigned long long ns);

// The test hook's tile (fd_debug_withhold_copies), INT_MAX where it is off.
int debug_withhold_tile();

// Streaming multiprocessors of a device (cached), and the library's own
// workspace of the paged attention for (device, stream): FD_* status codes.
int device_sm_count(int device, int* sms);
int paged_workspace(int device, cudaStream_t stream, size_t bytes, void** ptr);
void paged_release();

}  // namespace fd
