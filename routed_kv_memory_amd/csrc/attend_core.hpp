// attend_core.hpp -- what the attention over a paged local cache does whatever the cache's rows are held in:
// jobs, plans and their parts, the arithmetic on tiles of bf16 rows, and the join.
//
// The work is a list of jobs: a job is a set of columns (token, query head of one KV head; the G
// heads of a token side by side) over [c memory rows ; local rows p0 .. p1).  A sequence of many new
// tokens, or alone in its group, makes one job over everything; the others of a group make one job of
// all their tokens over the shared rows and one job each over its own rows.  Memory rows are visible to
// all columns of a job; of the local rows a column sees those below its own limit.  Lengths are on the
// device, so each workgroup forms the list itself (a few loads and two scans over the jobs, in LDS; calls of
// many workgroups do so once, attend_plan_kernel) and finds its part of it; the host only bounds the number
// of workgroups.
#pragma once

#include "msa_device.hpp"
#include "msa_kernels.hpp"

#include <type_traits>

namespace msa {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
// Columns of a wave that streams, and most of such a job.  Two such blocks in a wave take more registers than it
// has (a step of 16 samples, 32 columns of 8 share their rows: 205 against 164 us); the other way round, 16
// samples' own rows (4 columns each) as shared tiles take 254 against 166 us.
constexpr int kStreamCols = 16;
constexpr int kCols = 32;                 // columns of a wave that shares tiles
// A sequence of more columns than this does not share its group's rows: parts of so many columns cost
// more to write and join than the rows cost to read again (three sequences of 509 tokens, 32 heads, among 27 of
// one token over 1,500 shared rows: 195 us, 256 us sharing; from 128 to 512 it is the same).  Eight sequences over 4,000
// shared rows, two layers: 600 columns each 375 us, 459 sharing; 400 columns 278 us alone, 324 sharing as here.
constexpr int kAlone = 512;
constexpr int kWide = kWaves * kCols;     // columns of a workgroup of the second kind
constexpr int kBlockUnits = kCols / kStreamCols;    // units of the workspace that its waves' columns take
constexpr int kSets = kHeads / kWaves;    // head sets of a streamed job: streams of rows it makes
constexpr int kStreamRows = 32;           // rows of a streamed tile, in bf16
constexpr int kTileRows = 32;             // rows of a shared tile
// bf16 per staged row of a stream: 16-byte reads of 16 K rows, and transposed reads of 16 dims of
// 8 V rows, meet every LDS bank once
constexpr int kKStride = kDim + 8;
constexpr int kVStride = kDim + 16;
constexpr int kMaxSeqs = 2048;            // MSA_MAX_SEQS
constexpr int kSegments = 32;             // pieces of streams a workgroup lists at a time
// Two workgroups fit a CU (registers, LDS): 512 fill the chip.  A layer gets its share of them, but at
// least kBothWgs where there are jobs of both kinds: items come in eights (the heads), and a handful of
// eights would not split the work evenly.  16 samples of one question, 18 layers: 199 us with 28, 175 with 40,
// 173 with 56, 186 with 64, 182 with 72.  Others are within 6% from 28 to 80: 36 layers 298-332 us (least with 28, 314
// with 56), four questions in 12 layers 199-224 (least with 80, 210 with 56), a mixed batch in 18 layers 731-774.
constexpr int kWgs = 512;
constexpr int kBothWgs = 56;
// A call of more workgroups than this has its plans made once, in a launch before: 2,048 sequences of 16 rows behind
// 64 that each eight share, 18 layers, take 4.1 ms (14.3 with a plan in every workgroup); one token over 4,364
// rows would take 66 us, so 62.
constexpr int64_t kPlanWgs = 4096;

struct Plan;

struct AttendArgs {
  int32_t B, n_groups, n_q, Hq, G, g_shift, max_ctx, n_pages, page_shift, max_pages;
  const uint16_t* q;
  const int32_t *q_off, *grp_off;
  const uint16_t *ctx_k, *ctx_v;
  const int32_t* ctx_len;
  const void *k_pages, *v_pages;            // in the cache's format
  const int32_t *page_table, *kv_len, *pre_len;
  float scale2;                           // scale * log2 e
  void* out;
  int32_t wgs, both_wgs;                  // workgroups aimed at in a layer: jobs of one kind, of both
  int32_t unit_cols;                      // columns of a unit of the workspace: kStreamCols, or fewer if there are no more
  int32_t stream_units, max_units;        // units of one layer: of streamed parts, all
  int4* desc;                             // [L][n_q][own rows, shared rows][2]: where a token's parts are
  float2* ml;                             // [L][max_units][unit_cols], the parts: maximum (log2 units) and sum
  float* acc;                             // [L][max_units][unit_cols][128]
  Plan* plans;                            // [L][kThreads], or null: each workgroup makes its own
};

struct Job {
  int32_t t0, cols;        // first packed token, columns
  int32_t seq, grp;        // whose page table, whose memory rows
  int32_t c, p0, p1;       // memory rows, local rows [p0, p1)
  int32_t shared, split;   // the group's shared rows; own rows next to a shared job
};

// The lengths of one layer in LDS (in the memory of the tiles, before those come), clamped but for kv_len.
struct Lengths {
  int32_t *off, *grp;             // [kMaxSeqs + 1]
  int32_t *len, *clen, *pre;      // [kMaxSeqs]
  // bit b: sequence b shares rows with none before it (first of its group, alone, or behind one that is)
  uint32_t* start;                // [kMaxSeqs / 32 + 1]
  uint32_t* sums;                 // [8][kWaves]
  int4* items;                    // [kThreads]: of each job, where a thread has one at most
  bool grouped;                   // whether any sequence may share: not where each is its own group
};
constexpr int kStartWords = kMaxSeqs / 32 + 1;
constexpr int kStage = 1024;              // 16-byte words of a stage of shared tiles (below)

__device__ __forceinline__ Lengths lengths_in(u32x4* a, u32x4* b, u32x4* c, u32x4* d) {
  Lengths n;
  n.off = reinterpret_cast<int32_t*>(a);
  n.len = reinterpret_cast<int32_t*>(b);
  n.pre = n.len + kMaxSeqs;
  n.clen = reinterpret_cast<int32_t*>(c);
  n.grp = reinterpret_cast<int32_t*>(d);
  n.start = reinterpret_cast<uint32_t*>(n.off + kMaxSeqs + 4);
  n.sums = n.start + kStartWords + 3;
  n.items = reinterpret_cast<int4*>(n.clen + kMaxSeqs);
  n.grouped = false;
  return n;
}

__device__ __forceinline__ int32_t clampi(int32_t v, int32_t lo, int32_t hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Number of entries of the ascending a[1 .. n] that are <= v.
__device__ __forceinline__ int32_t count_upto(const int32_t* a, int32_t n, int32_t v) {
  int32_t lo = 0, hi = n;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (a[mid + 1] <= v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void load_lengths(const AttendArgs& a, Lengths& n, int64_t layer, int tid) {
  const bool grouped = a.grp_off != nullptr;
  bool own = a.n_groups == a.B;             // groups 0, 1, ... of one sequence each need no shared jobs
  const int32_t cap = a.max_pages << a.page_shift;
  for (int32_t i = tid; i <= a.B; i += kThreads) {
    n.off[i] = clampi(a.q_off[i], 0, a.n_q);
    if (i < a.B) n.len[i] = a.kv_len[i];
  }
  for (int32_t g = tid; g <= a.n_groups; g += kThreads) {
    if (grouped) {
      const int32_t at = clampi(a.grp_off[g], 0, a.B);
      n.grp[g] = at;
      own &= at == g;
    }
    if (g < a.n_groups) {
      n.clen[g] = a.max_ctx > 0 ? clampi(a.ctx_len[layer * a.n_groups + g], 0, a.max_ctx) : 0;
      n.pre[g] = grouped && a.pre_len ? clampi(a.pre_len[g], 0, cap) : 0;
    }
  }
  if (grouped)
    for (int i = tid; i < kStartWords; i += kThreads) n.start[i] = 0;
  n.grouped = !__syncthreads_and(own) && grouped;
  if (!n.grouped) return;
  auto mark = [&](int32_t b) { atomicOr(n.start + (b >> 5), 1u << (b & 31)); };
  for (int32_t g = tid; g <= a.n_groups; g += kThreads) mark(n.grp[g]);
  for (int32_t b = tid; b < a.B; b += kThreads)
    if ((n.off[b + 1] - n.off[b]) * a.G > kAlone) {
      mark(b);
      mark(b + 1);
    }
  if (tid == 0) mark(a.B);
  __syncthreads();
}

__device__ __forceinline__ bool starts(const Lengths& n, int32_t b) { return n.start[b >> 5] >> (b & 31) & 1; }

// The group of sequence b, n_groups for one outside all groups (it has no memory rows).
__device__ __forceinline__ int32_t group_of(const AttendArgs& a, const Lengths& n, int32_t b) {
  const int32_t g = count_upto(n.grp, a.n_groups, b);
  return g < a.n_groups && n.grp[g] <= b ? g : a.n_groups;
}

// Job b < B: sequence b's rows.  Job B + b, in groups: the rows that the sequences from b on share (b the
// first of them).
__device__ __forceinline__ Job job_of(const AttendArgs& a, const Lengths& n, int32_t j) {
  const bool grouped = n.grouped;
  Job x;
  const int32_t b = j < a.B ? j : j - a.B, cap = a.max_pages << a.page_shift;
  x.shared = j >= a.B;
  x.t0 = n.off[b];
  x.cols = 0;
  x.split = 0;
  x.seq = b;
  x.p0 = 0;
  if (!grouped) {
    x.cols = max(0, n.off[b + 1] - x.t0) * a.G;
    x.grp = b;
    x.c = n.clen[b];
    x.p1 = clampi(n.len[b], 0, cap);
    return x;
  }
  const bool first = starts(n, b), alone = first && starts(n, b + 1);
  if (x.shared && (!first || alone)) return x;
  const int32_t g = group_of(a, n, b);
  const bool in = g < a.n_groups;
  x.grp = in ? g : 0;
  x.c = in ? n.clen[g] : 0;
  const int32_t pre = in ? n.pre[g] : 0;
  if (x.shared) {
    if (x.c + pre == 0) return x;
    int32_t w = (b + 1) >> 5;               // the next start: B at the latest
    uint32_t bits = n.start[w] & (~0u << ((b + 1) & 31));
    while (!bits) bits = n.start[++w];
    x.seq = n.grp[g];
    x.p1 = pre;
    x.cols = max(0, n.off[32 * w + __builtin_ctz(bits)] - x.t0) * a.G;
    return x;
  }
  x.cols = max(0, n.off[b + 1] - x.t0) * a.G;
  x.p1 = clampi(n.len[b], 0, cap);
  if (!alone) {
    x.split = x.c + pre > 0;
    x.c = 0;
    x.p0 = pre;
  }
  return x;
}

// How a cache holds its local rows: the rows of a streamed tile, memory rows (always bf16) and local ones, what
// either tile costs, and whether a layer's longest items come first.
struct RowsBf16 {
  static constexpr int kStreamCtx = kStreamRows, kStreamLocal = kStreamRows, kCtxCost = 1, kLocalCost = 1;
  static constexpr bool kLongestFirst = false;
};

// Tiles: t memory rows each, then `local` local rows each; one for a job without rows (its columns are zero).
__device__ __forceinline__ int32_t ctx_tiles(const Job& x, int32_t t) { return (x.c + t - 1) / t; }
__device__ __forceinline__ int32_t tiles_of(const Job& x, int32_t t, int32_t local) {
  return max(1, ctx_tiles(x, t) + (max(0, x.p1 - x.p0) + local - 1) / local);
}
__device__ __forceinline__ int32_t item_tiles(const Job& x) { return tiles_of(x, kTileRows, kTileRows); }

// Cost of a stream's first t tiles, of all of them, and the first tile behind a cost.
template <class F>
__device__ __forceinline__ uint32_t stream_cost(const Job& x, int32_t t) {
  const int32_t c = min(t, ctx_tiles(x, F::kStreamCtx));
  return (uint32_t)(c * F::kCtxCost + (t - c) * F::kLocalCost);
}
template <class F>
__device__ __forceinline__ int32_t stream_tiles(const Job& x) { return tiles_of(x, F::kStreamCtx, F::kStreamLocal); }
template <class F>
__device__ __forceinline__ int32_t tile_behind(const Job& x, uint32_t cost) {
  const uint32_t c = ctx_tiles(x, F::kStreamCtx);
  return (int32_t)(cost <= c * F::kCtxCost ? (cost + F::kCtxCost - 1) / F::kCtxCost
                                           : c + (cost - c * F::kCtxCost + F::kLocalCost - 1) / F::kLocalCost);
}

// Keeps a uniform value in scalar registers: the compiler would rather load kernel arguments again in every
// tile, and wait for them.
template <typename T>
__device__ __forceinline__ T kept(T v) {
  asm("" : "+s"(v));
  return v;
}

// Row of the page pool of job row lr (a local row).
__device__ __forceinline__ int32_t page_row(const AttendArgs& a, int32_t seq, int32_t lr) {
  const int32_t page = clampi(a.page_table[(int64_t)seq * a.max_pages + (lr >> a.page_shift)], 0, a.n_pages - 1);
  return (page << a.page_shift) + (lr & ((1 << a.page_shift) - 1));
}

// Local rows that packed token t sees, of a sequence with `len` local rows (new ones included; not clamped)
// whose tokens end before off_next.
__device__ __forceinline__ int32_t visible_rows(int32_t len, int32_t off_next, int32_t t) {
  return len <= 0 ? 0 : len - (off_next - t) + 1;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  auto add = [&](uint32_t o) { v += o; };
  add(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));    // row_shr 1, 2, 4, 8
  add(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));    // row_bcast 15, 31
  add(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}

// Inclusive sums over the workgroup's threads of two counts, and their totals; `slot`: 0 or 1, the scans of one
// plan use different memory, so each needs one barrier.
__device__ __forceinline__ void scan2(const Lengths& n, int slot, uint32_t& x, uint32_t& y, uint32_t* all, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  uint32_t* sums = n.sums + 2 * kWaves * slot;
  x = wave_scan(x);
  y = wave_scan(y);
  if (lane == 63) {
    sums[2 * wave] = x;
    sums[2 * wave + 1] = y;
  }
  __syncthreads();
  all[0] = all[1] = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) {
      x += sums[2 * w];
      y += sums[2 * w + 1];
    }
    all[0] += sums[2 * w];
    all[1] += sums[2 * w + 1];
  }
}

// A wave's running state.  State: lane l holds column l & 31, dims 32 d + 8 (r >> 2) + 4 (l >> 5) + (r & 3) of
// it.  State16: column l & 15, dims 16 d + 4 (l >> 4) + r.
struct State {
  static constexpr int kBlocks = 4, kRegs = 16;
  float m, l, neg;     // neg: -m, 0 for no row so far
  f32x16 o[4];
};
struct State16 {
  static constexpr int kBlocks = 8, kRegs = 4;
  float m, l, neg;
  f32x4 o[8];
};

template <typename St>
__device__ __forceinline__ void clear(St& st) {
  st.m = -__builtin_huge_valf();
  st.l = st.neg = 0.f;
#pragma unroll
  for (int d = 0; d < St::kBlocks; ++d)
#pragma unroll
    for (int r = 0; r < St::kRegs; ++r) st.o[d][r] = 0.f;
}

__device__ __forceinline__ float halves_max(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(x[0]) + __uint_as_float(x[1]);
}

__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

// bits of the 16-bit halves of w that are infinities or NaN (0xFFFF each)
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma_of(u32x4 x, u32x4 y, f32x16 c) { return mfma32(x, y, c); }
__device__ __forceinline__ f32x4 mfma_of(u32x4 x, u32x4 y, f32x4 c) { return mfma16(x, y, c); }

// A V^T fragment with entries that are not finite, for a product with weights of which some are masked
// to 0 (0 * inf is NaN): the entries are taken out of it, and their kind is added to the output where
// a weight above 0 meets one.
template <typename Acc>
__device__ __forceinline__ u32x4 without_specials(u32x4 raw, u32x4 bad, u32x4 p, Acc& o) {
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    u32x4 one;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      auto is = [&](uint32_t x) {
        return kind == 0 ? x == 0x7F80u : (kind == 1 ? x == 0xFF80u : (x & 0x7FFFu) > 0x7F80u);
      };
      one[e] = (is(raw[e] & 0xFFFFu) ? 0x3F80u : 0u) | (is(raw[e] >> 16) ? 0x3F800000u : 0u);
    }
    Acc t;
#pragma unroll
    for (int r = 0; r < (int)(sizeof(Acc) / 4); ++r) t[r] = 0.f;
    t = mfma_of(one, p, t);
    const float add = kind == 0 ? __builtin_huge_valf() : (kind == 1 ? -__builtin_huge_valf() : __builtin_nanf(""));
#pragma unroll
    for (int r = 0; r < (int)(sizeof(Acc) / 4); ++r) o[r] += t[r] > 0.f ? add : 0.f;
  }
  return raw & ~bad;
}

// A masked row's weight is 0, but 0 * inf is NaN (and with probabilities in three parts, an infinity meets a
// residual of either sign).  A weight above 1 (below) may overflow with values near the largest, and a
// maximum beyond 2^29 is rounded by more than the weights' range bears.  So when what was summed up is not
// finite, or the maximum that large, it is gone through once more with CAREFUL set: V entries that are no finite
// numbers are taken out of the products, the maximum is always the largest score, and the scores are
// rounded as it is.

__device__ __forceinline__ f32x16 zeros16() {
  return f32x16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// Scores behind a column's first `left` of a tile's 32 rows to -inf.
__device__ __forceinline__ void mask_rows(f32x16& s, int32_t left, int h) {
  left -= 4 * h;
#pragma unroll
  for (int r = 0; r < 16; ++r) s[r] = 8 * (r >> 2) + (r & 3) < left ? s[r] : -__builtin_huge_valf();
}

__device__ __forceinline__ float max16(const f32x16& s) {
  float m = s[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) m = fmaxf(m, s[r]);
  return m;
}

// The running maximum (log2 units) against a tile's largest score: it is raised only when the tile passes it by
// more than 2^8, so most tiles skip the rescale (a prompt of 8,000 tokens 1.18 ms, 1.25 raising it always).
template <bool CAREFUL, typename St>
__device__ __forceinline__ void raise_to(float mt, float scale2, St& st) {
  const float ninf = -__builtin_huge_valf();
  mt *= scale2;
  const bool raise = mt > st.m + (CAREFUL ? 0.f : 8.f);
  if (__builtin_expect(__ballot(raise) != 0, 0)) {
    const float mn = raise ? mt : st.m;
    const float alpha = st.m == ninf ? (raise ? 0.f : 1.f) : __builtin_amdgcn_exp2f(st.m - mn);
    st.m = mn;
    st.neg = mn == ninf ? 0.f : -mn;
    st.l *= alpha;
#pragma unroll
    for (int d = 0; d < St::kBlocks; ++d) st.o[d] *= alpha;
  }
}

// A score's distance to the maximum.
template <bool CAREFUL>
__device__ __forceinline__ float below(float s, float scale2, float neg_m) {
#pragma clang fp contract(off)
  return CAREFUL ? s * scale2 + neg_m : __builtin_fmaf(s, scale2, neg_m);
}

// Probabilities of 8 scores as a B operand of the second product, and into the sum.
// PARTS 3 (fp32 output): three bf16 values, each the rounding of what those before it leave, together the fp32
// value but for 2^-25 of it.  Two leave 2^-17: 2.3e-6 of the output against 4.3e-7 with three, for 850
// against 985 us where the matrix cores bind (8 prompts of up to 1,088 tokens, 4 layers), next to nothing elsewhere.
// PARTS 1 (bf16 output): one bf16 value, whose rounding (2^-8 of each weight) is the size of the
// output's own; the sum is then taken of the rounded values, so the weights still add up to one.  The output is then
// off by 2.2e-3 (rms, relative; 1.7e-3 is the output's rounding alone).  Two parts take 1.46 ms where one takes 1.08 (the
// long prompt), 236 against 186 us in a mixed batch, and in streams 183 against 175 us (64 users).
template <int PARTS, bool CAREFUL>
__device__ __forceinline__ void weights(const float* s, float scale2, float neg_m, u32x4* pw, float& l) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p0 = __builtin_amdgcn_exp2f(below<CAREFUL>(s[2 * e], scale2, neg_m));
    const float p1 = __builtin_amdgcn_exp2f(below<CAREFUL>(s[2 * e + 1], scale2, neg_m));
    const uint32_t w = pack2_bf16(p0, p1);
    pw[0][e] = w;
    if (PARTS > 1) {
      l += p0 + p1;
      float r0 = p0 - __uint_as_float(w << 16), r1 = p1 - __uint_as_float(w & 0xFFFF0000u);
      pw[1][e] = pack2_bf16(r0, r1);
      if (PARTS > 2) {
        r0 -= __uint_as_float(pw[1][e] << 16);
        r1 -= __uint_as_float(pw[1][e] & 0xFFFF0000u);
        pw[PARTS - 1][e] = pack2_bf16(r0, r1);
      }
    } else {
      l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), l, false);
    }
  }
}

// O^T += V^T . P^T for one fragment of V^T.
template <int PARTS, bool CAREFUL, typename Acc>
__device__ __forceinline__ void add_values(u32x4 vf, const u32x4* pw, Acc& o) {
  if (CAREFUL) {
    u32x4 bad;
#pragma unroll
    for (int e = 0; e < 4; ++e) bad[e] = not_finite(vf[e]);
    if (__ballot((bad[0] | bad[1] | bad[2] | bad[3]) != 0)) vf = without_specials(vf, bad, pw[0], o);
  }
#pragma unroll
  for (int i = 0; i < PARTS; ++i) o = mfma_of(vf, pw[i], o);
}

template <typename St>
__device__ __forceinline__ bool needs_care(const St& st) {
  const float inf = __builtin_huge_valf();
  bool odd = st.m != -inf && __builtin_fabsf(st.m) >= 0x1p29f;
#pragma unroll
  for (int d = 0; d < St::kBlocks; ++d)
#pragma unroll
    for (int r = 0; r < St::kRegs; ++r) odd |= !(__builtin_fabsf(st.o[d][r]) < inf);
  return __ballot(odd) != 0;
}

__device__ __forceinline__ u32x4 frag_of(uint2 lo, uint2 hi) { return u32x4{lo.x, lo.y, hi.x, hi.y}; }

// A column of one head: whether there is one, its token and its row of q and out.
struct Column {
  bool live;
  int32_t t;
  int64_t row;
};

__device__ __forceinline__ Column column_of(const AttendArgs& a, const Job& x, int64_t layer, int head, int32_t col) {
  Column y;
  y.live = col < x.cols;
  const int32_t at = y.live ? col : 0;
  y.t = x.t0 + (at >> a.g_shift);
  y.row = (layer * a.n_q + y.t) * a.Hq + head * a.G + (at & (a.G - 1));
  return y;
}

// Four dims from `d` on of a column: into a part of the workspace (the index of its column there) or the output.
__device__ __forceinline__ void write_part(const AttendArgs& a, int64_t part, int d, float v0, float v1, float v2,
                                           float v3) {
  *reinterpret_cast<float4*>(a.acc + part * kDim + d) = make_float4(v0, v1, v2, v3);
}
template <bool BF16_OUT>
__device__ __forceinline__ void write_out(const AttendArgs& a, int64_t row, int d, float v0, float v1, float v2, float v3) {
  if (BF16_OUT)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kDim + d) =
        make_uint2(pack2_bf16(v0, v1), pack2_bf16(v2, v3));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kDim + d) = make_float4(v0, v1, v2, v3);
}

// The wave's columns: as a part of the workspace (unit >= 0) or as the output; `l` the column's whole sum.
template <bool BF16_OUT>
__device__ __forceinline__ void write_state(const AttendArgs& a, const State& st, float l, const Column& y, int64_t layer,
                                            int32_t unit, int lane) {
  const int c = lane & 31, h = lane >> 5;
  if (!y.live) return;
  const int64_t part = (layer * a.max_units + unit) * a.unit_cols + c;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (unit >= 0 && h == 0) a.ml[part] = make_float2(st.m, l);
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = st.o[d][4 * i], v1 = st.o[d][4 * i + 1], v2 = st.o[d][4 * i + 2], v3 = st.o[d][4 * i + 3];
      if (unit >= 0) write_part(a, part, 32 * d + 8 * i + 4 * h, v0, v1, v2, v3);
      else write_out<BF16_OUT>(a, y.row, 32 * d + 8 * i + 4 * h, v0 * inv, v1 * inv, v2 * inv, v3 * inv);
    }
}
template <bool BF16_OUT>
__device__ __forceinline__ void write_state(const AttendArgs& a, const State16& st, float l, const Column& y, int64_t layer,
                                            int32_t unit, int lane) {
  const int j = lane & 15, g = lane >> 4;
  if (!y.live) return;
  const int64_t part = (layer * a.max_units + unit) * a.unit_cols + j;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (unit >= 0 && g == 0) a.ml[part] = make_float2(st.m, l);
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    if (unit >= 0) write_part(a, part, 16 * d + 4 * g, st.o[d][0], st.o[d][1], st.o[d][2], st.o[d][3]);
    else write_out<BF16_OUT>(a, y.row, 16 * d + 4 * g, st.o[d][0] * inv, st.o[d][1] * inv, st.o[d][2] * inv,
                             st.o[d][3] * inv);
  }
}

// Where a token's parts are: part k of head h of a column is unit
//   first[h / kWaves] + (h % kWaves) * head_step + k * part_step,   k < parts[h / kWaves]
// and column `col` from its first on (up to 32, in two units).  The item that begins a job writes it for the job's tokens.
struct Parts {
  int32_t first[kSets], parts[kSets];
};
static_assert(kSets == 2, "a descriptor holds two head sets");

__device__ __forceinline__ void describe(const AttendArgs& a, const Job& x, const Column& y, int64_t layer,
                                         const Parts& p, int32_t add, int32_t head_step, int32_t part_step,
                                         int32_t col) {
  int4* d = a.desc + ((layer * a.n_q + y.t) * 2 + (x.shared ? 1 : 0)) * 2;
  d[0] = make_int4(p.first[0] + add, p.parts[0], p.first[1] + add, p.parts[1]);
  d[1] = make_int4(head_step, part_step, col, x.split);
}

// ------------------------------------------------------------------ who does what
//
// Streamed jobs make two streams of rows each, one for each set of 4 heads (a wave each).  All streams of
// a layer are laid end to end and cut into equal shares, one for each workgroup: every one has tiles of the same
// cost whatever the lengths are, and one start.  A share holds pieces of one or more
// streams; a piece is one part of its columns.
//
// The other jobs make items: a column block of 128, one head, a chunk of the rows.  A job's rows are cut
// into its share of the workgroups, rounded down, so that they all run at once (rounded to the nearest, 61
// sequences behind 30,000 shared rows take 140 us, so 118), but into chunks of eight tiles at least
// (four or sixteen measure the same).  Of a job's items those of the last column blocks, whose tokens see the most rows,
// come first (workgroups start in order); heads fastest (workgroups go to the 8 XCDs in turn: a
// head's rows stay in one L2).  Rows in 4 bits: jobs with longer items come first, and what the rounding down leaves of the
// workgroups goes to the longest (24 sequences of five drafted tokens and 100 to 9,000 rows: 127 us in the jobs' order, 119
// sorted and paired (attend4_kernel), 108 with those chunks too; the mixed batch 254 and 241).  Other lengths of drafted
// tokens: in 1 to 18 layers 57 to 332 us, 69 to 346 with none of the three; the chunks alone: two sequences in 18 layers 131 us (165
// without), 24 in two 118 (125), but 45 of 2,000 to 3,000 rows in one layer 74 (69.5).  The order costs streams alone 1 us.

__device__ __forceinline__ bool streamed(const Job& x) { return x.cols <= kStreamCols; }

// Chunks of an item job's rows; `aim` is workgroups per tile of work.
__device__ __forceinline__ int32_t chunks_of(const Job& x, float aim) {
  const int32_t t = item_tiles(x);
  return max(1, min(t / 8, (int32_t)((float)t * aim)));
}
__device__ __forceinline__ int32_t items_of(const Job& x) { return (x.cols + kWide - 1) / kWide * kHeads; }

// 32-column blocks of an item of so many columns.
__device__ __forceinline__ int32_t blocks_of(int32_t cols) { return cols <= kCols ? 1 : (cols <= 2 * kCols ? 2 : kWaves); }
// Units of the parts of one chunk of an item job: two for each 32-column block and head.
__device__ __forceinline__ int32_t units_of(const Job& x) {
  const int32_t whole = (x.cols - 1) / kWide;             // column blocks before the last
  return kHeads * kBlockUnits * (whole * kWaves + blocks_of(x.cols - whole * kWide));
}

struct Plan {
  int32_t j0, j1;                 // this thread's jobs
  Job first;                      // the first of them (mostly the only one)
  uint32_t cost, streams;         // of streamed jobs before them
  uint32_t items, units;          // items, and units of those that are parts, before them
  uint32_t all_cost, all_items, share, shares;     // cost of a share, shares
  int32_t more;                   // chunks of this thread's only job on top of chunks_of
  float aim;
};

template <class F>
__device__ __forceinline__ Plan make_plan(const AttendArgs& a, const Lengths& n, int tid) {
  Plan p;
  const int32_t nj = n.grouped ? 2 * a.B : a.B, per = (nj + kThreads - 1) / kThreads;
  p.j0 = min(nj, tid * per);
  p.j1 = min(nj, p.j0 + per);
  p.first.cols = 0;
  if (p.j0 < p.j1) p.first = job_of(a, n, p.j0);
  // the cost of a layer's streams fits 32 bits: 2 x 4,096 streams of at most 2^17 tiles of local rows (2^16 in 4 bits),
  // and memory rows, which fit the card.  Work of the items: fp32 sum of whole numbers, in the same order in every
  // workgroup
  uint32_t cost = 0, streams = 0, all[2];
  float work = 0.f;
  for (int32_t j = p.j0; j < p.j1; ++j) {
    const Job x = j == p.j0 ? p.first : job_of(a, n, j);
    if (x.cols == 0) continue;
    if (streamed(x)) {
      cost += kSets * stream_cost<F>(x, stream_tiles<F>(x));
      streams += kSets;
    } else {
      work += (float)item_tiles(x) * (float)items_of(x);
    }
  }
  p.cost = cost;
  p.streams = streams;
  work = wave_sum(work);
  float* sums = reinterpret_cast<float*>(n.sums + 4 * kWaves);
  if ((tid & 63) == 0) sums[tid >> 6] = work;
  // jobs with items, where a thread has one at most: how many, and this thread's place among them
  const bool own = F::kLongestFirst && nj <= kThreads && p.j0 < p.j1 && p.first.cols > 0 && !streamed(p.first);
  const uint64_t owners = __ballot(own);
  int32_t n_own = 0, at = __builtin_popcountll(owners & ((1ull << (tid & 63)) - 1));
  if ((tid & 63) == 0) n.sums[5 * kWaves + (tid >> 6)] = (uint32_t)__builtin_popcountll(owners);
  scan2(n, 0, cost, streams, all, tid);
  p.cost = cost - p.cost;
  p.streams = streams - p.streams;
  p.all_cost = all[0];
  work = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    work += sums[w];
    const int32_t c = (int32_t)n.sums[5 * kWaves + w];
    n_own += c;
    at += w < tid >> 6 ? c : 0;
  }
  p.all_items = p.items = p.units = 0;
  p.more = 0;
  p.aim = 0.f;
  p.shares = a.wgs;
  if (work > 0.f) {                               // uniform
    // a streamed tile is 4 heads' rows, an item's is one head's, of more columns: 4.2 against 1.2 us where
    // both wait for HBM, 2.3 against 1.2 next to items bound by the matrix cores (2, 3 and 4 in place of
    // one for the other measure the same within 3%)
    const float streams_work = 3.f / F::kLocalCost * (float)p.all_cost;
    const int32_t wgs = p.all_cost ? a.both_wgs : a.wgs;
    // 2^-10 below: the roundings of the sum
    p.aim = wgs * (1.f - 0x1p-10f) / (work + streams_work);
    uint32_t ahead = 0;
    if (n_own > 1) {                              // uniform
      // Longest items first, those of one length in the jobs' order.  A tile costs about 1 + column blocks.
      int32_t nch = own ? chunks_of(p.first, p.aim) : 0;
      const int32_t k = own ? items_of(p.first) : 0, t = own ? item_tiles(p.first) : 0;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        const int32_t length = own ? (t + nch - 1) / nch * (1 + blocks_of(p.first.cols)) : 0;
        if (own) n.items[at] = make_int4(length, nch * k, k, 0);
        __syncthreads();
        uint32_t total = 0, chunks = 0;           // all items; one chunk of each of those ahead
        ahead = 0;
#pragma unroll 4
        for (int32_t i = 0; i < n_own; ++i) {
          const int4 o = n.items[i];
          const bool first = o.x > length || (o.x == length && i < at);
          total += o.y;
          ahead += first ? o.y : 0;
          chunks += first ? o.z : 0;
        }
        // workgroups that the rounding down leaves: a chunk more for the longest
        if (pass > 0 || p.all_cost > 0 || total >= (uint32_t)wgs) break;      // uniform
        if (own && total + chunks + k <= (uint32_t)wgs && t / 8 > nch) p.more = 1;
        nch += p.more;
        __syncthreads();
      }
    }
    uint32_t items = 0, units = 0;
    for (int32_t j = p.j0; j < p.j1; ++j) {
      const Job x = j == p.j0 ? p.first : job_of(a, n, j);
      if (x.cols == 0 || streamed(x)) continue;
      const int32_t nch = chunks_of(x, p.aim) + p.more;
      const uint32_t k = nch * items_of(x);
      items += k;
      if (x.shared || x.split || nch > 1) units += nch * units_of(x);
    }
    p.items = items;
    p.units = units;
    scan2(n, 1, items, units, all, tid);
    p.items = n_own > 1 ? ahead : items - p.items;
    p.units = units - p.units;
    p.all_items = all[0];
    p.shares = max((int32_t)(streams_work * p.aim), wgs - (int32_t)min(p.all_items, (uint32_t)wgs));
    p.shares = p.all_cost ? max(p.shares, 1u) : 0u;
  }
  // a tile is of the share that its cost begins in: none between a stream's first and last is without one
  constexpr uint32_t least = F::kCtxCost > F::kLocalCost ? F::kCtxCost : F::kLocalCost;
  p.share = p.shares ? max(least, (p.all_cost + p.shares - 1) / p.shares) : least;
  return p;
}

// This thread's part of the layer's plan, from the launch before or made here.
template <class F>
__device__ __forceinline__ Plan plan_of(const AttendArgs& a, const Lengths& n, int64_t layer, int tid) {
  return a.plans ? a.plans[layer * kThreads + tid] : make_plan<F>(a, n, tid);
}

struct Segment {
  Job x;
  int32_t set, tile0, tile1;    // head set, tiles of the stream
  int32_t slot;                 // its parts' units are kWaves * slot ..; -1: writes the output
  int32_t first;                // begins the job
  int32_t limit0;               // local rows (from p0) that the job's first token sees, one more each token;
                                // shared jobs: searched for each token
  Parts parts;
};

// The pieces of streams in share `number`, from cost `from` of the layer's on: up to kSegments into `seg`, their
// number in n_seg[0]; returns where the list ends, 0 where that is the share's end.
template <class F>
__device__ __forceinline__ uint32_t list_segments(const AttendArgs& a, const Lengths& n, const Plan& p, Segment* seg,
                                                  uint32_t* n_seg, uint32_t number, uint32_t from) {
  const uint32_t share = p.share;
  const uint64_t begin = (uint64_t)number * share;
  if (begin >= p.all_cost) return 0;
  from = max(from, (uint32_t)begin);
  const uint32_t to = (uint32_t)min(begin + share, (uint64_t)p.all_cost);
  auto walk = [&](auto&& f) __attribute__((always_inline)) {
    uint32_t u = p.cost, s = p.streams;
    for (int32_t j = p.j0; j < p.j1 && u < to; ++j) {
      const Job x = j == p.j0 ? p.first : job_of(a, n, j);
      if (x.cols == 0 || !streamed(x)) continue;
      const int32_t tiles = stream_tiles<F>(x);
      const uint32_t t = stream_cost<F>(x, tiles), last = stream_cost<F>(x, tiles - 1);     // where the last tile begins
      for (int set = 0; set < kSets; ++set, u += t, ++s)
        if (u < to && u + last >= from) f(x, set, u, t, last, s);
    }
  };
  // the first stream with a tile that begins at `from` or behind it is the list's first
  walk([&](const Job&, int, uint32_t, uint32_t, uint32_t, uint32_t s) { atomicMax(n_seg + 1, ~s); });
  __syncthreads();
  const uint32_t s_first = ~n_seg[1];
  walk([&](const Job& x, int set, uint32_t u, uint32_t t, uint32_t last, uint32_t s) {
    const uint32_t k = s - s_first;
    if (k >= kSegments) return;
    Segment& g = seg[k];
    g.x = x;
    g.set = set;
    g.tile0 = tile_behind<F>(x, max(from, u) - u);
    g.tile1 = tile_behind<F>(x, min(to, u + t) - u);
    g.first = set == 0 && g.tile0 == 0;
    g.limit0 = visible_rows(n.len[x.seq], n.off[x.seq + 1], x.t0) - x.p0;
    // the stream's tiles lie in shares w0 .. w1; stream + share number is a number of its own for every
    // piece, consecutive along a stream
    bool whole = true;
    for (int v = 0; v < kSets; ++v) {
      const uint32_t u0 = u + (v - set) * t, w0 = u0 / share, w1 = (u0 + last) / share;
      g.parts.first[v] = (int32_t)(kWaves * (w0 + s + v - set));
      g.parts.parts[v] = (int32_t)(w1 - w0 + 1);
      if (w1 > w0) whole = false;
    }
    const bool direct = whole && !x.shared && !x.split;
    if (direct) g.parts.first[0] = g.parts.first[1] = -1;
    g.slot = direct ? -1 : (int32_t)(number + s);
    // only offsets that are not ascending make more parts than there is room for
    if (g.slot >= 0 && kWaves * (g.slot + 1) > a.stream_units) g.x.cols = 0;
    atomicMax(n_seg, k + 1);
    if (k == kSegments - 1) n_seg[2] = min(to, u + t);
  });
  __syncthreads();
  // a full list may end with the share, also inside a stream
  return n_seg[0] < kSegments || n_seg[2] >= to ? 0 : n_seg[2];
}

struct Item {
  Job x;
  int32_t valid, nch, tile0, tile1;     // chunks of the job's tiles, this item's tiles
  int32_t head, col0, blocks;           // first column, column blocks (1, 2 or 4)
  int32_t unit, width, first;           // its first unit (-1: writes the output), units; first chunk and head
  Parts parts;
};

__device__ __forceinline__ void find_item(const AttendArgs& a, const Lengths& n, const Plan& p, Item& it, uint32_t id,
                                          int tid) {
  if (tid == 0) it.valid = 0;
  __syncthreads();
  uint32_t at = p.items, u = p.units;
  for (int32_t j = p.j0; j < p.j1 && at <= id; ++j) {
    const Job x = j == p.j0 ? p.first : job_of(a, n, j);
    if (x.cols == 0 || streamed(x)) continue;
    const int32_t nch = chunks_of(x, p.aim) + p.more, ncb = items_of(x) / kHeads;
    const uint32_t k = nch * ncb * kHeads;
    const bool parts = x.shared || x.split || nch > 1;
    if (id < at + k) {
      const int32_t i = (int32_t)(id - at), t = item_tiles(x);
      const int32_t chunk = i / kHeads % nch, xb = i / kHeads / nch, len = (t + nch - 1) / nch;
      it.x = x;
      it.nch = nch;
      it.head = i % kHeads;
      it.col0 = (ncb - 1 - xb) * kWide;
      it.blocks = blocks_of(x.cols - it.col0);
      it.tile0 = min(t, chunk * len);
      it.tile1 = min(t, it.tile0 + len);
      it.first = chunk == 0 && it.head == 0;
      // units lie as the items do: by column block from the last (the only one that may be narrower), chunk and head
      const int32_t width = kBlockUnits * it.blocks, narrow = kBlockUnits * blocks_of(x.cols - (ncb - 1) * kWide);
      const int64_t begin = a.stream_units + (int64_t)u +
                            (xb ? nch * kHeads * (narrow + (xb - 1) * (int64_t)(kBlockUnits * kWaves)) : 0);
      const int64_t unit = begin + (chunk * kHeads + it.head) * width;
      it.width = width;
      it.unit = parts ? (int32_t)unit : -1;
      for (int v = 0; v < kSets; ++v) {
        it.parts.first[v] = parts ? (int32_t)begin + v * kWaves * width : -1;
        it.parts.parts[v] = nch;
      }
      // only offsets that are not ascending make more parts than there is room for
      it.valid = !parts || unit + width <= a.max_units;
      break;
    }
    at += k;
    if (parts) u += nch * units_of(x);
  }
  __syncthreads();
}

// ------------------------------------------------------------------ tiles of up to 16 columns

// 32 rows whose scores are formed (rows 16 kb + 4 g + r of column j in s[kb][r]) and whose V rows lie in the wave's tile.
template <int PARTS, bool CAREFUL>
__device__ __forceinline__ void attend_scored(const uint16_t* tile, const f32x4* s, int32_t left, float scale2, int lane,
                                              State16& st) {
  const int j = lane & 15, g = lane >> 4;
  // probabilities as the B operand: k slot 8 g + e holds row 4 g + e (e < 4) or 16 + 4 g + e - 4
  float v[8], mt = -__builtin_huge_valf();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 16 * (e >> 2) + 4 * g + (e & 3) < left ? s[e >> 2][e & 3] : -__builtin_huge_valf();
    mt = fmaxf(mt, v[e]);
  }
  raise_to<CAREFUL>(rows4_max(mt), scale2, st);
  u32x4 pw[PARTS];
  weights<PARTS, CAREFUL>(v, scale2, st.neg, pw, st.l);
  // a 16-lane group reads 16 dims of 4 rows transposed
  const uint16_t* vsrc = tile + (4 * g + (j >> 2)) * kVStride + 4 * (j & 3);
#pragma unroll
  for (int d = 0; d < 8; ++d)
    add_values<PARTS, CAREFUL>(frag_of(lds_read_tr16(vsrc + 16 * d), lds_read_tr16(vsrc + 16 * kVStride + 16 * d)), pw,
                               st.o[d]);
}

// 16 rows whose scores are formed: the other half of the product's k axis holds nothing.
template <int PARTS, bool CAREFUL>
__device__ __forceinline__ void attend_scored16(const uint16_t* tile, f32x4 s, int32_t left, float scale2, int lane,
                                                State16& st) {
  const int j = lane & 15, g = lane >> 4;
  float v[8], mt = -__builtin_huge_valf();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = e < 4 && 4 * g + (e & 3) < left ? s[e & 3] : -__builtin_huge_valf();
    mt = fmaxf(mt, v[e]);
  }
  raise_to<CAREFUL>(rows4_max(mt), scale2, st);
  u32x4 pw[PARTS];
  weights<PARTS, CAREFUL>(v, scale2, st.neg, pw, st.l);
  const uint16_t* vsrc = tile + (4 * g + (j >> 2)) * kVStride + 4 * (j & 3);
#pragma unroll
  for (int d = 0; d < 8; ++d)
    add_values<PARTS, CAREFUL>(frag_of(lds_read_tr16(vsrc + 16 * d), make_uint2(0u, 0u)), pw, st.o[d]);
}

// 32 rows in the wave's tile: K rows while the scores are formed, then V rows; `then` once these are in.
template <int PARTS, bool CAREFUL, typename Then>
__device__ __forceinline__ void attend_rows(uint16_t* tile, const u32x4* pv, const u32x4* qf, int32_t left, float scale2,
                                            int lane, State16& st, Then&& then) {
  const int j = lane & 15, g = lane >> 4;
  f32x4 s[2];
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    s[kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < 4; ++d)
      s[kb] = mfma16(*reinterpret_cast<const u32x4*>(tile + (16 * kb + j) * kKStride + 32 * d + 8 * g), qf[d], s[kb]);
  }
  // the wave's LDS accesses complete in order: the V rows may follow the reads
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<u32x4*>(tile + (4 * i + g) * kVStride + 8 * j) = pv[i];
  then();
  attend_scored<PARTS, CAREFUL>(tile, s, left, scale2, lane, st);
}

// ------------------------------------------------------------------ tiles of more columns

// A stage holds 32 K rows, then 32 V rows, 16 chunks of 16 bytes each, as the direct
// global -> LDS loads write them: lane l of load i brings chunk (l & 15) of row 4 i + (l >> 4).  The
// chunks of a row are permuted (bf16 rows: by the lanes' source addresses), so that fragment reads meet every bank
// once: chunk x of K row r lies at x ^ (r & 15) (16 rows, one chunk each), of V row r at
// x ^ 5 (r & 3) (4 rows, 4 chunks each).  16 lanes that write a chunk of four rows' four blocks of 32 dims meet
// every bank once as well.
static_assert(kStage == 2 * kTileRows * 16, "K rows and V rows");

typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// A stage chosen at run time.
__device__ __forceinline__ uint32_t lds_at(u32x4* p) { return (uint32_t)(uintptr_t)(lptr_t)p; }
__device__ __forceinline__ const u32x4* lds_ptr(uint32_t at) {
  return (const u32x4*)(__attribute__((address_space(3))) const u32x4*)(uintptr_t)at;
}

// This lane's pieces of K and V fragments in a stage, as byte offsets.  The compiler is kept from knowing how they
// come about: it then adds a stage's address in the instruction and not in registers for each stage.
struct StageReads {
  int kb[8], vb[4];
  __device__ __forceinline__ explicit StageReads(int lane) {
    const int c = lane & 31, h = lane >> 5, i = lane & 15;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      kb[d] = 16 * (c * 16 + ((2 * d + h) ^ (c & 15)));
      asm("" : "+v"(kb[d]));
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int x = 4 * (d ^ (i >> 2)) + ((2 * ((lane >> 4) & 1) + ((i >> 1) & 1)) ^ (i >> 2));
      vb[d] = 2 * ((kTileRows + 4 * h + (i >> 2)) * kDim + 8 * x + 4 * (i & 1));
      asm("" : "+v"(vb[d]));
    }
  }
  // row c, chunk 2 d + h
  __device__ __forceinline__ u32x4 k(const u32x4* stage, int d) const {
    return *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(stage) + kb[d]);
  }
  // dims 32 d .. of rows 16 m + 4 h + 0..3 and 16 m + 8 + 4 h + 0..3
  __device__ __forceinline__ u32x4 v(const u32x4* stage, int m, int d) const {
    const char* p = reinterpret_cast<const char*>(stage) + vb[d] + 32 * m * kDim;
    return frag_of(lds_read_tr16(reinterpret_cast<const uint16_t*>(p)),
                   lds_read_tr16(reinterpret_cast<const uint16_t*>(p + 16 * kDim)));
  }
};

// The rows of N stages, tiles t and t + 1, into the state; a column sees the first left(tile) of them (whole: all of
// both).  Two at once make one decision about the maximum for 64 rows, and the second tile's scores are formed while
// the first one's settle.  kf: the K fragments of a single tile where they have been read already.
template <int PARTS, bool CAREFUL, int N, typename Left>
__device__ __forceinline__ void attend_tiles(const u32x4* kf, const u32x4* stage_a, const u32x4* stage_b,
                                             const StageReads& at, const u32x4* qf, int32_t t, bool whole, Left&& left,
                                             float scale2, int h, State& st) {
  f32x16 s[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    s[u] = zeros16();
#pragma unroll
    for (int d = 0; d < 8; ++d) s[u] = mfma32(kf ? kf[d] : at.k(u ? stage_b : stage_a, d), qf[d], s[u]);
  }
  u32x4 vf[2][4];               // on their way while the softmax runs
  if (!CAREFUL) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int d = 0; d < 4; ++d) vf[m][d] = at.v(stage_a, m, d);
  }
  if (!whole) {
    asm volatile("" ::: );      // a branch: most tiles are whole, and selects for all would cost what the exps do
    mask_rows(s[0], left(t), h);
    if (N == 2) mask_rows(s[N - 1], left(t + 1), h);
  }
  float top = max16(s[0]);
  if (N == 2) top = fmaxf(top, max16(s[N - 1]));
  raise_to<CAREFUL>(halves_max(top), scale2, st);
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      // k slot 8 h + e holds row 16 m + 4 h + e (e < 4) or 16 m + 8 + 4 h + e - 4
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = s[u][8 * m + e];
      u32x4 pw[PARTS];
      weights<PARTS, CAREFUL>(v, scale2, st.neg, pw, st.l);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        add_values<PARTS, CAREFUL>(CAREFUL || u ? at.v(u ? stage_b : stage_a, m, d) : vf[m][d], pw, st.o[d]);
    }
}

struct ItemShared {
  Item item;
  int32_t most[kWaves];                   // local rows that a wave's columns see
  int32_t least[kWaves];                  // and that all of them see
  float m[kWaves][kCols], l[kWaves][kCols];
};

// An item's end: the states of the waves that share a column block joined, then written.
template <bool BF16_OUT>
__device__ __forceinline__ void finish_item(const AttendArgs& a, ItemShared& z, State& st, const Column& y, int64_t layer,
                                            int32_t unit, int32_t blocks, int cb, int32_t turn, int wave, int lane,
                                            u32x4* stage1, u32x4* stage2, u32x4* stage3) {
  const int c = lane & 31, h = lane >> 5;
  float l = halves_sum(st.l);
  if (blocks < kWaves) {       // join the states of a block's waves, in the first of them
    auto state_of = [&](int w) { return reinterpret_cast<float*>(w == 1 ? stage1 : (w == 2 ? stage2 : stage3)); };
    static_assert(kStage * 16 >= kCols * kDim * 4, "a wave's state fits");
    if (turn > 0) {
      if (h == 0) {
        z.m[wave][c] = st.m;
        z.l[wave][c] = l;
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(state_of(wave) + 4 * (c + kCols * (8 * d + 2 * i + h))) =
              make_float4(st.o[d][4 * i], st.o[d][4 * i + 1], st.o[d][4 * i + 2], st.o[d][4 * i + 3]);
    }
    __syncthreads();
    if (turn > 0) return;
    for (int w = wave + blocks; w < kWaves; w += blocks) {
      const float* o = state_of(w);
      const float m = fmaxf(st.m, z.m[w][c]), base = m == -__builtin_huge_valf() ? 0.f : m;
      const float f = __builtin_amdgcn_exp2f(st.m - base), g = __builtin_amdgcn_exp2f(z.m[w][c] - base);
      st.m = m;
      l = l * f + z.l[w][c] * g;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          st.o[d][r] = st.o[d][r] * f + g * o[4 * (c + kCols * (8 * d + 2 * (r >> 2) + h)) + (r & 3)];
    }
  }
  write_state<BF16_OUT>(a, st, l, y, layer, unit < 0 ? -1 : unit + kBlockUnits * cb, lane);
}

// The plans of all layers.
template <class F>
__global__ void __launch_bounds__(kThreads)
attend_plan_kernel(const AttendArgs a) {
  __shared__ u32x4 s0[kStage], s1[kStage], s2[kStage], s3[kStage];
  Lengths n = lengths_in(s0, s1, s2, s3);
  load_lengths(a, n, blockIdx.x, threadIdx.x);
  a.plans[blockIdx.x * (int64_t)kThreads + threadIdx.x] = make_plan<F>(a, n, threadIdx.x);
}

// Joins the parts of a token's own rows and of its group's shared rows: four dims of one query head
// a thread, the parts in order with a running maximum.
// A workgroup takes 8 heads of `per` tokens, of which it first looks up which have parts at all.  Latency is all
// here: the first token's descriptors are asked for at once with that, and own and shared parts together.
template <bool BF16_OUT>
__global__ void __launch_bounds__(256)
attend_join_kernel(const AttendArgs a, int32_t per) {
  const int64_t layer = blockIdx.z;
  const int32_t t0 = blockIdx.x * per;
  const int lane = threadIdx.x & 63;
  const int32_t hq = blockIdx.y * 8 + (threadIdx.x >> 5), d4 = 4 * (threadIdx.x & 31);
  const int32_t head = hq / a.G, hh = hq % a.G, set = head / kWaves;
  const int4* descs = a.desc + layer * a.n_q * 4;
  int4 d[4];                                // own rows' descriptor, the shared rows'
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = descs[(int64_t)t0 * 4 + i];
  const int32_t first_unit = descs[(int64_t)min(t0 + lane, a.n_q - 1) * 4].x;
  // the sequences' tokens: those before and behind have no descriptor, or what an earlier call left there
  const int32_t tb = clampi(a.q_off[0], 0, a.n_q), tn = min(t0 + per, clampi(a.q_off[a.B], 0, a.n_q));
  // per <= 64; a token whose first set has parts has parts of every set
  uint64_t todo = __ballot(t0 + lane >= tb && t0 + lane < tn && first_unit >= 0);
  for (; todo; todo &= todo - 1) {
    const int32_t t = t0 + __builtin_ctzll(todo);
    if (t != t0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = descs[(int64_t)t * 4 + i];
    }
    // parts 0 .. n[0] are the own rows', from there to n[0] + n[1] the shared rows'
    int32_t n[2];
    int64_t at[2], step[2];
    bool ok = true;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int4 d0 = d[2 * which], d1 = d[2 * which + 1];
      n[which] = 0;
      at[which] = step[which] = 0;
      if (which == 1 && d[1].w == 0) continue;
      const int32_t first = set ? d0.z : d0.x, parts = set ? d0.w : d0.y, col = d1.z + hh;
      const int64_t unit = first + (int64_t)(head % kWaves) * d1.x, end = unit + (int64_t)(parts - 1) * d1.y;
      // holds for every token of a sequence; offsets that are not ascending may leave a token without parts
      ok &= first >= 0 && parts >= 1 && parts <= a.max_units && d1.x >= 0 && d1.x <= kBlockUnits * kWaves && d1.y >= 0 &&
            col >= 0 && col < kCols && end < a.max_units && end * a.unit_cols + col < (int64_t)a.max_units * a.unit_cols;
      n[which] = parts;
      at[which] = (layer * a.max_units + unit) * a.unit_cols + col;
      step[which] = (int64_t)d1.y * a.unit_cols;
    }
    if (!ok) continue;
    const int32_t all = n[0] + n[1];
    float m = -__builtin_huge_valf(), l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < all; k0 += 8) {
      float2 ml[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int32_t k = min(k0 + u, all - 1);
        const int64_t p = k < n[0] ? at[0] + k * step[0] : at[1] + (k - n[0]) * step[1];
        ml[u] = a.ml[p];
        v[u] = *reinterpret_cast<const float4*>(a.acc + p * kDim + d4);
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < 8; ++u) mn = fmaxf(mn, ml[u].x);
      const float base = mn == -__builtin_huge_valf() ? 0.f : mn;     // no row so far
      const float s = __builtin_amdgcn_exp2f(m - base);
      l *= s;
      o.x *= s;
      o.y *= s;
      o.z *= s;
      o.w *= s;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (k0 + u >= all) continue;
        const float w = __builtin_amdgcn_exp2f(ml[u].x - base);
        l += w * ml[u].y;
        o.x += w * v[u].x;
        o.y += w * v[u].y;
        o.z += w * v[u].z;
        o.w += w * v[u].w;
      }
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = ((layer * a.n_q + t) * a.Hq + hq) * kDim + d4;
    if (BF16_OUT)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row) =
          make_uint2(pack2_bf16(o.x * inv, o.y * inv), pack2_bf16(o.z * inv, o.w * inv));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row) =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
}

// Bounds for one layer.  Shares: the workgroups aimed at, one more next to items.  Streamed pieces: one for each
// share and one more for each stream.  An item job of n > 16 columns has 8 ceil(n / 128) items a chunk, at most n / 2
// (8 at 17, 16 at 129) and 8 + n / 16; the items of jobs cut into more chunks and the shares are together
// at most the workgroups aimed at, and one.  Parts come from items of jobs that are cut (8 units of 16 columns at most),
// and in groups from all items of the shared rows and of the own rows next to them: of sequences of up to kAlone
// columns, two or more in a run of a group that shares.  Their columns are rounded up to 32, 64 or 128 at a job's
// end, to less than twice as many and 63 more at most: in 8 heads up to n units and up to n / 2 + 32.
struct Sizes {
  int32_t wgs, both_wgs, grid, unit_cols, stream_units, max_units;
  size_t desc, ml, acc, plans, total;
};

Sizes sizes_of(int64_t L, int64_t B, int64_t n_groups, int64_t n_q, int64_t G, bool grouped) {
  Sizes z;
  auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  const int64_t cols = n_q * G, shared_cols = grouped ? least(cols, kAlone * B) : 0, all_cols = cols + shared_cols;
  z.wgs = (int32_t)(L < kWgs ? kWgs / L : 1);
  z.both_wgs = z.wgs > kBothWgs ? z.wgs : kBothWgs;
  // every sequence with tokens, and the shared rows of two or more of a group or behind one on its own
  const int64_t jobs = least(B, n_q) + (grouped ? least(n_groups + cols / kAlone, least(B / 2, n_q)) : 0);
  const int64_t aimed = cols > kStreamCols ? z.both_wgs + 1 : z.wgs;
  const int64_t whole = cols > kStreamCols ? least(all_cols / 2, kHeads * jobs + all_cols / 16) : 0;
  const int64_t parts = cols > kStreamCols ? kBlockUnits * kWaves * aimed + least(2 * shared_cols, 32 * jobs + shared_cols) : 0;
  z.grid = (int32_t)(aimed + whole);
  z.unit_cols = (int32_t)least(cols, kStreamCols);
  z.stream_units = (int32_t)(kWaves * (aimed + kSets * jobs));
  z.max_units = (int32_t)(z.stream_units + parts);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  z.desc = up((size_t)L * n_q * 4 * sizeof(int4));
  z.ml = up((size_t)L * z.max_units * z.unit_cols * sizeof(float2));
  z.acc = up((size_t)L * z.max_units * z.unit_cols * kDim * sizeof(float));
  z.plans = L * z.grid > kPlanWgs ? up((size_t)L * kThreads * sizeof(Plan)) : 0;
  z.total = z.desc + z.ml + z.acc + z.plans;
  return z;
}

// Groups cannot share anything between fewer than two sequences.
inline bool can_share(int32_t B) { return B > 1; }

// `kernel`: attend_kernel of this output type, over rows held as F.
template <class F, bool BF16_OUT>
void launch_as(void (*kernel)(const AttendArgs), const AttendArgs& a, const Sizes& z, int32_t L, hipStream_t s) {
  if (a.plans) hipLaunchKernelGGL(attend_plan_kernel<F>, dim3((unsigned)L), dim3(kThreads), 0, s, a);
  const unsigned most = 32768, y = (unsigned)z.grid < most ? (unsigned)z.grid : most;    // a launch's y may have 65,535
  hipLaunchKernelGGL(kernel, dim3((unsigned)L, y, (z.grid + y - 1) / y), dim3(kThreads), 0, s, a);
  // a workgroup for 8 heads of one token, of several (at most 64) where there are many
  const int64_t rows = (int64_t)a.n_q * a.G * L;
  const int32_t per = (int32_t)(rows < 8192 ? 1 : (rows > 64 * 8192 ? 64 : rows / 8192));
  hipLaunchKernelGGL(attend_join_kernel<BF16_OUT>, dim3((unsigned)((a.n_q + per - 1) / per), (unsigned)a.G, (unsigned)L),
                     dim3(256), 0, s, a, per);
}

inline AttendArgs args_of(const Sizes& z, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* q,
                          const int32_t* q_off, const int32_t* grp_off, const uint16_t* ctx_k, const uint16_t* ctx_v,
                          const int32_t* ctx_len, int32_t max_ctx, const void* k_pages, const void* v_pages,
                          int32_t n_pages, int32_t page_shift, const int32_t* page_table, int32_t max_pages,
                          const int32_t* kv_len, const int32_t* pre_len, float scale, void* out, void* ws) {
  char* w = static_cast<char*>(ws);
  return {B, n_groups, n_q, Hq, Hq / kHeads, __builtin_ctz(Hq / kHeads), max_ctx, n_pages, page_shift, max_pages, q, q_off,
          grp_off, ctx_k, ctx_v, ctx_len, k_pages, v_pages, page_table, kv_len, pre_len, scale * 1.4426950408889634f, out,
          z.wgs, z.both_wgs, z.unit_cols, z.stream_units, z.max_units, reinterpret_cast<int4*>(w),
          reinterpret_cast<float2*>(w + z.desc), reinterpret_cast<float*>(w + z.desc + z.ml),
          z.plans ? reinterpret_cast<Plan*>(w + z.desc + z.ml + z.acc) : nullptr};
}

}  // namespace
}  // namespace msa
