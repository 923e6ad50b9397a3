// read4.hip -- rows of a paged local cache held in 4 bits back as packed bf16 rows.
//
// Packed row t (i-th of sequence b's) is local row row0[b] + i of b: row r % P of page page_table[b][r / P], each
// code as the bf16 value it stands for (cache4.hpp).
//
// One wave takes one row in one layer: 8 lanes a head, 16 dims each.
#include "cache4.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

constexpr int kReadWaves = 4;              // rows per workgroup

__global__ void __launch_bounds__(64 * kReadWaves)
read4_kernel(int32_t B, int32_t n_rows, const int32_t* __restrict__ row_off, const int32_t* __restrict__ row0,
             const int32_t* __restrict__ page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
             const uint8_t* __restrict__ k_pages, const uint8_t* __restrict__ v_pages, uint16_t* __restrict__ k_out,
             uint16_t* __restrict__ v_out) {
  const int lane = threadIdx.x & 63;
  const int32_t t = blockIdx.x * kReadWaves + (threadIdx.x >> 6);
  const int64_t layer = blockIdx.y;
  if (t >= n_rows) return;                  // whole waves; no barrier below
  const int32_t b = seq_of_token(row_off, B, t, lane);
  if (b >= B) return;                       // rows behind the last sequence are left as they are
  const int32_t q0 = row_off[b];
  if (t < q0 || t >= row_off[b + 1]) return;          // offsets that are not ascending
  const int64_t row = (int64_t)(row0 ? row0[b] : 0) + (t - q0);
  int32_t page = -1;
  if (row >= 0 && (row >> page_shift) < max_pages) page = page_table[(int64_t)b * max_pages + (row >> page_shift)];
  const bool have = page >= 0 && page < n_pages;
  const int64_t from = ((layer * n_pages + (have ? page : 0)) << page_shift) * kRow4;
  const int head = lane >> 3, j = lane & 7, r = (int)(row & ((1 << page_shift) - 1));
  const int64_t at = (layer * n_rows + t) * kRow + head * kDim + 16 * j;
  const int64_t codes = from + codes4_at(head, r, page_shift) + 8 * j;
  const int64_t scale = from + scales4_at(head, r, page_shift) + (j >> 1);
  auto put = [&](const uint8_t* pages, uint16_t* out) {
    u32x4 lo = {0u, 0u, 0u, 0u}, hi = lo;   // no such row
    if (have) {
      const uint2 w = *reinterpret_cast<const uint2*>(pages + codes);
      const float s = scale4(pages[scale]);
      lo = values4(w.x, s);
      hi = values4(w.y, s);
    }
    *reinterpret_cast<u32x4*>(out + at) = lo;
    *reinterpret_cast<u32x4*>(out + at + 8) = hi;
  };
  put(k_pages, k_out);
  put(v_pages, v_out);
}

}  // namespace

hipError_t launch_read4(int32_t L, int32_t B, int32_t n_rows, const int32_t* row_off, const int32_t* row0,
                        const int32_t* page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
                        const uint8_t* k_pages, const uint8_t* v_pages, uint16_t* k_out, uint16_t* v_out,
                        hipStream_t s) {
  hipLaunchKernelGGL(read4_kernel, dim3((unsigned)((n_rows + kReadWaves - 1) / kReadWaves), (unsigned)L),
                     dim3(64 * kReadWaves), 0, s, B, n_rows, row_off, row0, page_table, max_pages, page_shift, n_pages,
                     k_pages, v_pages, k_out, v_out);
  return hipGetLastError();
}

}  // namespace msa
