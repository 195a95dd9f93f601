// kvc_cache.h -- structures shared by the host half of libkvc and the kernels
// of the resident 8-bit cache (kvc_cache_rows.hip, kvc_attend.hip).  Not part
// of the public ABI (include/kvc.h is).
#pragma once
#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "kvc.h"

namespace kvc {

// The cache and the batch of a call, as the kernels see them.
struct CacheView {
  uint8_t *k_codes, *v_codes;               // [page][head][token][D], [page][head][D][token]
  float *k_scales, *v_scales;               // [page][head]
  uint32_t stride_page, stride_scale;       // bytes; floats
  uint32_t num_pages, heads, tshift;        // tokens_per_page = 1 << tshift
};
struct BatchView {
  const int32_t *table, *cu, *lengths;
  uint32_t* flags;                          // may be null
  int64_t stride_table;
  uint32_t n_seqs, n_rows, max_rows, max_len;
  // Work units of the launch: unit u belongs to sequence u / per_seq when
  // per_seq is not 0, else to the last sequence whose first unit,
  // cu[b] * unit_mul / unit_div + b * unit_add, is at most u (seq_of_unit).
  uint32_t per_seq, unit_mul, unit_div, unit_add;
};
struct RowsView {
  uint16_t* data;                           // [row][head][D]
  int64_t stride_row, stride_head;          // elements
};

struct RowsParams {                         // write, read
  CacheView c;
  BatchView b;
  RowsView k, v;
  uint32_t units;                           // page units
};

struct AttendParams {
  CacheView c;
  BatchView b;
  RowsView q, out;
  float* lse;                               // [row][query head], may be null
  float* ws;                                // splits > 1: partial sums, then (max, sum) pairs
  uint32_t dtype, group;                    // group = query heads of a KV head
  uint32_t causal, window;
  float scale_log2;                         // softmax scale * log2(e)
  uint32_t units;                           // row tiles
  uint32_t splits, chunk;                   // context splits of `chunk` tokens each
  uint32_t turn_at, turn;                   // attend_rows_kernel's order of tiles: [at, 2 at) turned by so many
  BatchView join;                           // splits > 1: units are rows
  uint32_t join_units;
};
constexpr uint32_t kMaxSplits = 2048;
// attend_rows_kernel: waves of a workgroup, workgroups that a CU holds (by LDS
// and registers), query rows of a workgroup (32 a wave, 16 at D = 256).  At
// D <= 64 two workgroups of eight waves work while the other one waits at its
// barrier: two 4096-row prompts of 32 heads of 64 take 209 us, 512-row chunks
// over 16,000 positions 310; with one workgroup of twelve it was 219 and 512,
// with one of sixteen 195 and 331, but 171 against 144 for 16 x 1024 rows.
// D = 256: twelve waves are no faster (101 us against 103, 52 against 46 for 64 rows).
constexpr int attend_row_waves(int d) { return d == 128 ? 12 : 8; }
constexpr int attend_row_resident(int d) { return d <= 64 ? 2 : 1; }
constexpr int attend_tile_rows(int d) { return attend_row_waves(d) * (d == 256 ? 16 : 32); }

// Launchers.  Weak, so that the host half links without the kernels, as the
// tests of its argument checks build it; a call then reports KVC_E_HIP.
__attribute__((weak)) hipError_t launch_cache_write(const RowsParams& p, uint32_t codec, uint32_t dtype,
                                                    uint32_t head_dim, hipStream_t stream);
__attribute__((weak)) hipError_t launch_cache_read(const RowsParams& p, uint32_t codec, uint32_t dtype,
                                                   uint32_t head_dim, hipStream_t stream);
__attribute__((weak)) hipError_t launch_cache_attend(const AttendParams& p, uint32_t codec, uint32_t head_dim,
                                                     uint32_t tile_rows, hipStream_t stream);

}  // namespace kvc
