// read4.hip -- rows of a paged local cache held in 4 bits back as packed bf16 rows.
//
// Packed row t (i-th of sequence b's) is local row row0[b] + i of b: row r % P of page page_table[b][r / P], each
// code as the bf16 value it stands for (cache4.hpp).
//
// Bound: HBM, nearly all of it what is written (5,184 bytes a row and layer, 4,096 of them out): 540,000 rows take 528 us
// (5.3 TB/s), a few rows 8 us.  One wave takes one row in one layer; lane l holds dims 8 l .. and 512 + 8 l .. of its
// 8 x 128, so each store of the wave is 1 KiB without gaps (16 dims a lane, two stores of every other 16 bytes: 609 us where
// this takes 415, ragged conversations).  Several rows a wave, looked up at once, are slower: 555 us with two, 604 with four; 333 rows in 18
// layers 8.2 us with one, 9.3 with four.
#include "cache4.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

constexpr int kReadWaves = 4;              // rows of a workgroup

__global__ void __launch_bounds__(64 * kReadWaves)
read4_kernel(int32_t B, int32_t n_rows, const int32_t* __restrict__ row_off, const int32_t* __restrict__ row0,
             const int32_t* __restrict__ page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
             const uint8_t* __restrict__ k_pages, const uint8_t* __restrict__ v_pages, uint16_t* __restrict__ k_out,
             uint16_t* __restrict__ v_out) {
  const int lane = threadIdx.x & 63;
  const int32_t t = __builtin_amdgcn_readfirstlane(blockIdx.x * kReadWaves + (threadIdx.x >> 6));
  const int64_t layer = blockIdx.y;
  if (t >= n_rows) return;                  // whole waves; no barrier below
  const int32_t b = __builtin_amdgcn_readfirstlane(seq_of_token(row_off, B, t, lane));
  if (b >= B) return;                       // rows behind the last sequence are left as they are
  const int32_t q0 = row_off[b];
  if (t < q0 || t >= row_off[b + 1]) return;          // offsets that are not ascending
  const int64_t row = (int64_t)(row0 ? row0[b] : 0) + (t - q0);
  int32_t page = -1;
  if (row >= 0 && (row >> page_shift) < max_pages) page = page_table[(int64_t)b * max_pages + (row >> page_shift)];
  const bool have = page >= 0 && page < n_pages;
  const int64_t from = ((layer * n_pages + page) << page_shift) * kRow4;
  const int r = (int)(row & ((1 << page_shift) - 1));
  const int d = lane & 15;                  // dims 8 d .. of heads lane >> 4 and 4 + (lane >> 4)
  uint32_t codes[4] = {0u, 0u, 0u, 0u}, scales[4] = {0u, 0u, 0u, 0u};      // zeros: no such row
  if (have) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int head = 4 * h + (lane >> 4);
      const int64_t c = from + codes4_at(head, r, page_shift) + 4 * d, s = from + scales4_at(head, r, page_shift) + (d >> 2);
      codes[h] = *reinterpret_cast<const uint32_t*>(k_pages + c);
      codes[2 + h] = *reinterpret_cast<const uint32_t*>(v_pages + c);
      scales[h] = k_pages[s];
      scales[2 + h] = v_pages[s];
    }
  }
  const int64_t to = (layer * n_rows + t) * kRow + 8 * lane;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    *reinterpret_cast<u32x4*>(k_out + to + 512 * h) = values4(codes[h], scale4(scales[h]));
    *reinterpret_cast<u32x4*>(v_out + to + 512 * h) = values4(codes[2 + h], scale4(scales[2 + h]));
  }
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
