// attend.hip -- attention of ragged new tokens over [memory context ; paged local rows], the
// context and the first local pages shared by the sequences of a group.
//
// For every layer, token i of sequence b (n_b new tokens) in group g sees the group's memory rows
// 0 .. ctx_len[g]) and its local rows 0 .. kv_len[b] - n_b + i; query head hq reads KV head
// hq / (Hq / 8); the output is the softmax-weighted sum of the visible V rows.
//
// One wave per (query head, token, layer): lane i holds dims 2 i and 2 i + 1, rows one by one with
// a running maximum and sum.
#include "msa_device.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

template <bool BF16_OUT>
__global__ void __launch_bounds__(64)
attend_kernel(int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* __restrict__ q,
              const int32_t* __restrict__ q_off, const int32_t* __restrict__ grp_off,
              const uint16_t* __restrict__ ctx_k, const uint16_t* __restrict__ ctx_v,
              const int32_t* __restrict__ ctx_len, int32_t max_ctx, const uint16_t* __restrict__ k_pages,
              const uint16_t* __restrict__ v_pages, int32_t n_pages, int32_t page_shift,
              const int32_t* __restrict__ page_table, int32_t max_pages, const int32_t* __restrict__ kv_len,
              float scale, void* __restrict__ out) {
  const int lane = threadIdx.x;
  const int32_t hq = blockIdx.x, t = blockIdx.y;
  const int64_t layer = blockIdx.z;
  const int32_t b = seq_of_token(q_off, B, t, lane);
  if (b >= B) return;
  const int32_t q1 = q_off[b + 1];
  if (t < q_off[b] || t >= q1) return;
  int32_t g = b;
  if (grp_off) {
    g = 0;
    while (g < n_groups && !(grp_off[g] <= b && b < grp_off[g + 1])) ++g;
  }
  int32_t clen = max_ctx > 0 && g < n_groups ? ctx_len[layer * n_groups + g] : 0;
  clen = clen < 0 ? 0 : (clen > max_ctx ? max_ctx : clen);
  const int64_t cap = (int64_t)max_pages << page_shift;
  int64_t vis = (int64_t)kv_len[b] - (q1 - t) + 1;
  vis = vis < 0 ? 0 : (vis > cap ? cap : vis);

  const int kvh = hq / (Hq / kHeads);
  const int64_t at = ((layer * n_q + t) * Hq + hq) * kDim + 2 * lane;
  const uint32_t qw = *reinterpret_cast<const uint32_t*>(q + at);
  const float q0 = bf16_lo(qw), qh = bf16_hi(qw);
  float m = -__builtin_huge_valf(), l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int64_t r = 0; r < clen + vis; ++r) {
    const uint16_t *kr, *vr;
    if (r < clen) {
      const int64_t off = ((layer * n_groups + g) * max_ctx + r) * kRow;
      kr = ctx_k + off;
      vr = ctx_v + off;
    } else {
      const int32_t lr = (int32_t)(r - clen);
      int32_t page = page_table[(int64_t)b * max_pages + (lr >> page_shift)];
      page = page < 0 ? 0 : (page >= n_pages ? n_pages - 1 : page);
      const int64_t off = (((layer * n_pages + page) << page_shift) + (lr & ((1 << page_shift) - 1))) * kRow;
      kr = k_pages + off;
      vr = v_pages + off;
    }
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(kr + kvh * kDim + 2 * lane);
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(vr + kvh * kDim + 2 * lane);
    const float s = wave_sum(q0 * bf16_lo(kw) + qh * bf16_hi(kw)) * scale;
    const float mn = fmaxf(m, s);
    const float a = m == mn ? 1.f : __expf(m - mn), p = __expf(s - mn);
    l = l * a + p;
    o0 = o0 * a + p * bf16_lo(vw);
    o1 = o1 * a + p * bf16_hi(vw);
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (BF16_OUT)
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at) = pack2_bf16(o0 * inv, o1 * inv);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = make_float2(o0 * inv, o1 * inv);
}

}  // namespace

size_t attend_workspace_bytes(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq) { return 256; }

hipError_t launch_attend(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* q,
                         const int32_t* q_off, const int32_t* grp_off, const uint16_t* ctx_k, const uint16_t* ctx_v,
                         const int32_t* ctx_len, int32_t max_ctx, const uint16_t* k_pages, const uint16_t* v_pages,
                         int32_t n_pages, int32_t page_shift, const int32_t* page_table, int32_t max_pages,
                         const int32_t* kv_len, const int32_t* pre_len, float scale, bool bf16_out, void* out,
                         void* ws, hipStream_t s) {
  const dim3 grid((unsigned)Hq, (unsigned)n_q, (unsigned)L);
  if (bf16_out)
    hipLaunchKernelGGL(attend_kernel<true>, grid, dim3(64), 0, s, B, n_groups, n_q, Hq, q, q_off, grp_off, ctx_k, ctx_v,
                       ctx_len, max_ctx, k_pages, v_pages, n_pages, page_shift, page_table, max_pages, kv_len, scale, out);
  else
    hipLaunchKernelGGL(attend_kernel<false>, grid, dim3(64), 0, s, B, n_groups, n_q, Hq, q, q_off, grp_off, ctx_k, ctx_v,
                       ctx_len, max_ctx, k_pages, v_pages, n_pages, page_shift, page_table, max_pages, kv_len, scale, out);
  return hipGetLastError();
}

}  // namespace msa
