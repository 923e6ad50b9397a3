// attend.hip -- attention of ragged new tokens over [memory context ; paged local rows], the
// context and the first local pages shared by the sequences of a group.
//
// For every layer, token i of sequence b (n_b new tokens) in group g sees the group's memory rows
// 0 .. ctx_len[g]) and its local rows 0 .. kv_len[b] - n_b + i; query head hq reads KV head
// hq / (Hq / 8); the output is the softmax-weighted sum of the visible V rows.
//
// The work is a list of jobs: a job is a set of columns (token, query head of one KV head; the G
// heads of a token side by side) over [c memory rows ; local rows p0 .. p1).  A group of several
// sequences makes one job of all its tokens over the shared rows and one job for each sequence over
// its own rows; a sequence alone in its group makes one job over everything.  Memory rows are
// visible to all columns of a job; of the local rows a column sees those below its own limit.
// Lengths are on the device, so each workgroup forms the list itself (a few loads and two scans over
// the jobs, in LDS) and finds its part of it; the host only bounds the numbers of workgroups.
//
// A wave always holds 32 columns.  On the matrix cores (v_mfma_f32_32x32x16_bf16), per 32 rows:
// S^T = K . Q^T with K as the A operand and the columns as the B operand (registers), so lane l has
// column l & 31 and the rows 8 i + 4 (l >> 5) + 0..3; the softmax needs one exchange between the
// two halves of the wave.  For O^T += V^T . P^T the MFMA's k axis is taken in the order in which the
// scores already lie in the lanes, and V^T comes from the row-major tile by transposed LDS reads.
//
// Two kernels share the jobs by their columns:
// - up to 32 columns the rows' bytes bound the time (attend_stream_kernel): a wave takes one KV head
//   and streams rows through tiles of its own in LDS, without barriers;
// - more columns are bound by the matrix cores and the softmax's vector work (attend_tile_kernel): the
//   waves of a workgroup take one head and share each tile of 64 rows.
// Parts of a column's rows are joined by a third kernel; what is whole in one part is written directly.
#include "msa_device.hpp"
#include "msa_kernels.hpp"

#include <type_traits>

namespace msa {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCols = 32;                 // columns of a wave
constexpr int kWide = kWaves * kCols;     // columns of a workgroup of the tile kernel
constexpr int kSets = kHeads / kWaves;    // head sets of a streamed job: streams of rows it makes
constexpr int kStreamRows = 32;           // rows of a streamed tile
constexpr int kTileRows = 64;             // rows of a shared tile
// bf16 per staged row: 16-byte reads of 16 K rows, and transposed reads of 16 dims of 2 x 4 V rows, meet
// every LDS bank once
constexpr int kStride = kDim + 8;
constexpr int kVStride = kDim + 32;
constexpr int kMaxSeqs = 2048;            // MSA_MAX_SEQS
constexpr int kSegments = 32;             // pieces of streams a workgroup lists at a time
// Workgroups of one call: two of either kernel fit a CU (LDS and registers), 512 fill the chip.
constexpr int kStreamWgs = 512;
constexpr int kTileItems = 512;

struct AttendArgs {
  int32_t B, n_groups, n_q, Hq, G, max_ctx, n_pages, page_shift, max_pages;
  const uint16_t* q;
  const int32_t *q_off, *grp_off;
  const uint16_t *ctx_k, *ctx_v;
  const int32_t* ctx_len;
  const uint16_t *k_pages, *v_pages;
  const int32_t *page_table, *kv_len, *pre_len;
  float scale2;                           // scale * log2 e
  void* out;
  int32_t stream_wgs, tile_items;         // workgroups of the stream kernel, items aimed at by the other; a layer
  int32_t unit_cols;                      // columns of a part in the workspace
  int32_t stream_units, max_units;        // parts of one layer: the stream kernel's, all
  int4* desc;                             // [L][n_q][own rows, shared rows][2]: where a token's parts are
  float2* ml;                             // [L][max_units][unit_cols]: maximum (log2 units) and sum
  float* acc;                             // [L][max_units][unit_cols][128]
};

struct Job {
  int32_t t0, cols;        // first packed token, columns
  int32_t seq, grp;        // whose page table, whose memory rows
  int32_t c, p0, p1;       // memory rows, local rows [p0, p1)
  int32_t shared, split;   // the group's shared rows; own rows next to a shared job
};

// The lengths of one layer, clamped, in LDS (in the memory of the tiles, before those come).
struct Lengths {
  int32_t *off, *len, *grp;       // [kMaxSeqs + 1] each
  int32_t *clen, *pre;            // [kMaxSeqs]
  long long* sums;                // [kWaves][2]
};
constexpr int kLengthsA = 3 * (kMaxSeqs + 4) * 4, kLengthsB = 2 * kMaxSeqs * 4 + kWaves * 2 * 8;   // bytes

__device__ __forceinline__ Lengths lengths_in(void* a, void* b) {
  Lengths n;
  n.off = static_cast<int32_t*>(a);
  n.len = n.off + kMaxSeqs + 4;
  n.grp = n.len + kMaxSeqs + 4;
  n.clen = static_cast<int32_t*>(b);
  n.pre = n.clen + kMaxSeqs;
  n.sums = reinterpret_cast<long long*>(n.pre + kMaxSeqs);
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

__device__ __forceinline__ void load_lengths(const AttendArgs& a, const Lengths& n, int64_t layer, int tid) {
  const bool grouped = a.grp_off != nullptr;
  const int32_t cap = a.max_pages << a.page_shift;
  for (int32_t i = tid; i <= a.B; i += kThreads) {
    n.off[i] = clampi(a.q_off[i], 0, a.n_q);
    if (i < a.B) n.len[i] = clampi(a.kv_len[i], 0, cap);
  }
  for (int32_t g = tid; g <= a.n_groups; g += kThreads) {
    if (grouped) n.grp[g] = clampi(a.grp_off[g], 0, a.B);
    if (g < a.n_groups) {
      n.clen[g] = a.max_ctx > 0 ? clampi(a.ctx_len[layer * a.n_groups + g], 0, a.max_ctx) : 0;
      n.pre[g] = grouped && a.pre_len ? clampi(a.pre_len[g], 0, cap) : 0;
    }
  }
  __syncthreads();
}

// Jobs 0 .. n_groups) are the groups' shared rows (none when every sequence is its own group), then
// one for each sequence.
__device__ __forceinline__ Job job_of(const AttendArgs& a, const Lengths& n, int32_t j) {
  const bool grouped = a.grp_off != nullptr;
  const int32_t ng = grouped ? a.n_groups : 0;
  Job x;
  x.t0 = 0;
  x.cols = 0;
  x.split = 0;
  x.shared = j < ng;
  if (x.shared) {
    const int32_t s0 = n.grp[j], s1 = n.grp[j + 1];
    x.seq = s0;
    x.grp = j;
    x.c = n.clen[j];
    x.p0 = 0;
    x.p1 = n.pre[j];
    if (s1 - s0 < 2 || x.c + x.p1 == 0) return x;
    x.t0 = n.off[s0];
    x.cols = max(0, n.off[s1] - x.t0) * a.G;
    return x;
  }
  const int32_t b = j - ng;
  x.seq = b;
  x.t0 = n.off[b];
  x.cols = max(0, n.off[b + 1] - x.t0) * a.G;
  x.p0 = 0;
  x.p1 = n.len[b];
  if (!grouped) {
    x.grp = b;
    x.c = n.clen[b];
    return x;
  }
  const int32_t g = count_upto(n.grp, a.n_groups, b);
  const bool in = g < a.n_groups && n.grp[g] <= b;   // a sequence outside all groups has no memory rows
  x.grp = in ? g : 0;
  x.c = in ? n.clen[g] : 0;
  if (in && n.grp[g + 1] - n.grp[g] > 1) {
    x.p0 = n.pre[g];
    x.split = x.c + x.p0 > 0;
    x.c = 0;
  }
  return x;
}

// Tiles of t rows: those of the memory rows, then those of the local rows; one for a job without rows
// (its columns are zero).
__device__ __forceinline__ int32_t ctx_tiles(const Job& x, int32_t t) { return (x.c + t - 1) / t; }
__device__ __forceinline__ int32_t tiles_of(const Job& x, int32_t t) {
  return max(1, ctx_tiles(x, t) + (max(0, x.p1 - x.p0) + t - 1) / t);
}

// Row of the page pool of job row lr (a local row).
__device__ __forceinline__ int32_t page_row(const AttendArgs& a, int32_t seq, int32_t lr) {
  const int32_t page = clampi(a.page_table[(int64_t)seq * a.max_pages + (lr >> a.page_shift)], 0, a.n_pages - 1);
  return (page << a.page_shift) + (lr & ((1 << a.page_shift) - 1));
}

// Visible local rows of token t of sequence b (kv_len <= 0: none).
__device__ __forceinline__ int32_t visible_rows(const AttendArgs& a, int32_t b, int32_t off_next, int32_t t) {
  const int32_t len = a.kv_len[b];
  return len <= 0 ? 0 : len - (off_next - t) + 1;
}

template <typename T>
__device__ __forceinline__ T scan_incl(T v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}

// Inclusive scan over the workgroup's threads of two counts; their totals in `all`.
__device__ __forceinline__ void scan2(const Lengths& n, long long& x, long long& y, long long* all, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  x = scan_incl(x, lane);
  y = scan_incl(y, lane);
  __syncthreads();
  if (lane == 63) {
    n.sums[2 * wave] = x;
    n.sums[2 * wave + 1] = y;
  }
  __syncthreads();
  all[0] = all[1] = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) {
      x += n.sums[2 * w];
      y += n.sums[2 * w + 1];
    }
    all[0] += n.sums[2 * w];
    all[1] += n.sums[2 * w + 1];
  }
}

// A wave's running state: lane l holds column l & 31; dims 32 d + 8 (r >> 2) + 4 (l >> 5) + (r & 3) of it.
struct State {
  float m, l;
  f32x16 o[4];
};

__device__ __forceinline__ void clear(State& st) {
  st.m = -__builtin_huge_valf();
  st.l = 0.f;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) st.o[d][r] = 0.f;
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

// A V^T fragment with entries that are not finite, for a product with weights of which some are masked
// to 0 (0 * inf is NaN): the entries are taken out of it, and their kind is added to the output where
// a weight above 0 meets one.
__device__ __forceinline__ u32x4 without_specials(u32x4 raw, u32x4 bad, u32x4 p, f32x16& o) {
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
    f32x16 t = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    t = mfma32(one, p, t);
    const float add = kind == 0 ? __builtin_huge_valf() : (kind == 1 ? -__builtin_huge_valf() : __builtin_nanf(""));
#pragma unroll
    for (int r = 0; r < 16; ++r) o[r] += t[r] > 0.f ? add : 0.f;
  }
  return raw & ~bad;
}

// A masked row's weight is 0, but 0 * inf is NaN (and with probabilities in two parts, an infinity meets a
// residual of either sign).  So when what was summed up holds NaN, it is gone through once more with
// CAREFUL set, where V entries that are no finite numbers are taken out of the products: that gives
// what the columns see and nothing else.

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

// The running maximum (log2 units) against a tile's largest score: it is raised only when the tile passes
// it by more than 2^8, so most tiles skip the rescale.
__device__ __forceinline__ void raise_to(float mt, float scale2, State& st) {
  const float ninf = -__builtin_huge_valf();
  mt = halves_max(mt) * scale2;
  const bool raise = mt > st.m + 8.f;
  if (__builtin_expect(__ballot(raise) != 0, 0)) {
    const float mn = raise ? mt : st.m;
    const float alpha = st.m == ninf ? (raise ? 0.f : 1.f) : __builtin_amdgcn_exp2f(st.m - mn);
    st.m = mn;
    st.l *= alpha;
#pragma unroll
    for (int d = 0; d < 4; ++d) st.o[d] *= alpha;
  }
}

// Probabilities of 16 rows (half m of a tile's scores) as the B operand of a product, and into the sum:
// k slot 8 h + e holds row 16 m + 4 h + e (e < 4) or 16 m + 8 + 4 h + e - 4.
// PARTS: 2 gives a bf16 high part and a bf16 residual, 1 one bf16 value, whose rounding (2^-9 of each
// weight) is the size of a bf16 output's own; the sum is then taken of the rounded values, so the
// weights still add up to one.
template <int PARTS>
__device__ __forceinline__ void weights(const f32x16& s, int m, float scale2, float neg_m, u32x4& ph, u32x4& pl, float& l) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * m + 2 * e], scale2, neg_m));
    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * m + 2 * e + 1], scale2, neg_m));
    const uint32_t w = pack2_bf16(p0, p1);
    ph[e] = w;
    if (PARTS == 2) {
      pl[e] = pack2_bf16(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xFFFF0000u));
      l += p0 + p1;
    } else {
      l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), l, false);
    }
  }
}

// O^T += V^T . P^T for one 32-dim block and 16 rows.
template <int PARTS, bool CAREFUL>
__device__ __forceinline__ void add_values(u32x4 vf, const u32x4& ph, const u32x4& pl, f32x16& o) {
  if (CAREFUL) {
    u32x4 bad;
#pragma unroll
    for (int e = 0; e < 4; ++e) bad[e] = not_finite(vf[e]);
    if (__ballot((bad[0] | bad[1] | bad[2] | bad[3]) != 0)) vf = without_specials(vf, bad, ph, o);
  }
  o = mfma32(vf, ph, o);
  if (PARTS == 2) o = mfma32(vf, pl, o);
}

__device__ __forceinline__ bool holds_nan(const State& st) {
  bool odd = false;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd |= st.o[d][r] != st.o[d][r];
  return __ballot(odd) != 0;
}

__device__ __forceinline__ u32x4 frag_of(uint2 lo, uint2 hi) { return u32x4{lo.x, lo.y, hi.x, hi.y}; }

// 32 rows (padded tiles kt, vt in LDS) into the state of the wave's 32 columns.
template <int PARTS, bool CAREFUL>
__device__ __forceinline__ void attend32(const uint16_t* kt, const uint16_t* vt, const u32x4* qf, int32_t left,
                                         float scale2, int lane, State& st) {
  const int c = lane & 31, h = lane >> 5, i = lane & 15;
  f32x16 s = zeros16();
#pragma unroll
  for (int d = 0; d < 8; ++d)
    s = mfma32(*reinterpret_cast<const u32x4*>(kt + c * kStride + 16 * d + 8 * h), qf[d], s);
  mask_rows(s, left, h);
  raise_to(max16(s), scale2, st);
  const float neg_m = st.m == -__builtin_huge_valf() ? 0.f : -st.m;
  // a 16-lane group reads 16 dims of 4 rows transposed
  const uint16_t* vsrc = vt + (4 * h + (i >> 2)) * kVStride + 16 * ((lane >> 4) & 1) + 4 * (i & 3);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    u32x4 ph, pl;
    weights<PARTS>(s, m, scale2, neg_m, ph, pl, st.l);
#pragma unroll
    for (int d = 0; d < 4; ++d)
      add_values<PARTS, CAREFUL>(frag_of(lds_read_tr16(vsrc + 16 * m * kVStride + 32 * d),
                                       lds_read_tr16(vsrc + (16 * m + 8) * kVStride + 32 * d)),
                               ph, pl, st.o[d]);
  }
}

// The wave's columns of one head: whether there is a column, its token and its row of q and out.
struct Column {
  bool live;
  int32_t t;
  int64_t row;
};

__device__ __forceinline__ Column column_of(const AttendArgs& a, const Job& x, int64_t layer, int head, int32_t col) {
  Column y;
  y.live = col < x.cols;
  y.t = x.t0 + (y.live ? col / a.G : 0);
  y.row = (layer * a.n_q + y.t) * a.Hq + head * a.G + (y.live ? col % a.G : 0);
  return y;
}

__device__ __forceinline__ void load_q(const AttendArgs& a, const Column& y, int h, u32x4* qf) {
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    qf[d] = u32x4{0u, 0u, 0u, 0u};
    if (y.live) qf[d] = *reinterpret_cast<const u32x4*>(a.q + y.row * kDim + 16 * d + 8 * h);
  }
}

// The wave's columns: as a part of the workspace (unit >= 0) or as the output.
template <bool BF16_OUT>
__device__ __forceinline__ void write_state(const AttendArgs& a, State& st, const Column& y, int64_t layer, int32_t unit,
                                            int lane) {
  const int c = lane & 31, h = lane >> 5;
  const float l = halves_sum(st.l);
  if (!y.live) return;
  if (unit < 0) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = y.row * kDim + 32 * d + 8 * i + 4 * h;
        const float v0 = st.o[d][4 * i] * inv, v1 = st.o[d][4 * i + 1] * inv, v2 = st.o[d][4 * i + 2] * inv,
                    v3 = st.o[d][4 * i + 3] * inv;
        if (BF16_OUT)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack2_bf16(v0, v1), pack2_bf16(v2, v3));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v0, v1, v2, v3);
      }
  } else {
    const int64_t part = (layer * a.max_units + unit) * a.unit_cols + c;
    if (h == 0) a.ml[part] = make_float2(st.m, l);
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(a.acc + part * kDim + 32 * d + 8 * i + 4 * h) =
            make_float4(st.o[d][4 * i], st.o[d][4 * i + 1], st.o[d][4 * i + 2], st.o[d][4 * i + 3]);
  }
}

// Where a token's parts are: part k of head h of a column is unit
//   first[h / kWaves] + (h % kWaves) * head_step + k * part_step,   k < parts[h / kWaves]
// and column `col` of it.  The item that begins a job writes it for the job's tokens.
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

// ------------------------------------------------------------------ up to 32 columns
//
// A job makes two streams of rows, one for each set of 4 heads (a wave each).  All streams of a layer
// are laid end to end and cut into equal shares, one for each workgroup: every workgroup has the same
// number of tiles whatever the lengths are, and one start.  A share holds pieces of one or more
// streams; a piece is one part of its columns.

struct Segment {
  Job x;
  int32_t set, tile0, tile1;    // head set, tiles of the stream
  int32_t slot;                 // its parts' units are kWaves * slot ..; -1: writes the output
  int32_t first;                // begins the job
  Parts parts;
};

// The jobs of at most 32 columns whose streams reach into tiles [from, to) of the layer's: up to
// kSegments pieces into `seg`; returns where the list ends, in `n_seg` its length.
__device__ int64_t list_segments(const AttendArgs& a, const Lengths& n, Segment* seg, int32_t* n_seg, int64_t layer,
                                 int64_t from, int tid) {
  load_lengths(a, n, layer, tid);
  const int32_t nj = a.B + (a.grp_off ? a.n_groups : 0);
  const int32_t per = (nj + kThreads - 1) / kThreads, j0 = min(nj, tid * per), j1 = min(nj, j0 + per);
  long long tiles = 0, streams = 0, all[2];
  for (int32_t j = j0; j < j1; ++j) {
    const Job x = job_of(a, n, j);
    if (x.cols == 0 || x.cols > kCols) continue;
    tiles += kSets * tiles_of(x, kStreamRows);
    streams += kSets;
  }
  const long long my_tiles = tiles, my_streams = streams;
  scan2(n, tiles, streams, all, tid);
  const int64_t share = max(1LL, (all[0] + a.stream_wgs - 1) / a.stream_wgs);
  const int64_t begin = blockIdx.x * share;
  if (from < begin) from = begin;
  const int64_t to = min(begin + share, (int64_t)all[0]);
  // number of the stream that holds tile `from`, so that pieces get consecutive places in the list
  int64_t at = tiles - my_tiles, stream = streams - my_streams;
  if (tid == 0) {
    n_seg[0] = 0;
    n_seg[1] = 0;
  }
  __syncthreads();
  auto walk = [&](auto&& f) {
    int64_t u = at, s = stream;
    for (int32_t j = j0; j < j1; ++j) {
      if (u >= to) break;
      const Job x = job_of(a, n, j);
      if (x.cols == 0 || x.cols > kCols) continue;
      const int32_t t = tiles_of(x, kStreamRows);
      for (int set = 0; set < kSets; ++set, u += t, ++s)
        if (u < to && u + t > from) f(x, set, u, t, s);
    }
  };
  if (from < to)
    walk([&](const Job&, int, int64_t u, int32_t, int64_t s) {
      if (u <= from) n_seg[1] = (int32_t)s;
    });
  __syncthreads();
  const int32_t s_first = n_seg[1];
  if (from < to)
    walk([&](const Job& x, int set, int64_t u, int32_t t, int64_t s) {
      const int64_t k = s - s_first;
      if (k >= kSegments) return;
      Segment& g = seg[k];
      g.x = x;
      g.set = set;
      g.tile0 = (int32_t)(max(from, u) - u);
      g.tile1 = (int32_t)(min(to, u + t) - u);
      g.first = set == 0 && g.tile0 == 0;
      // the stream's tiles lie in shares w0 .. w1; place + share number is a number of its own for
      // every piece, consecutive along a stream
      bool whole = true;
      for (int v = 0; v < kSets; ++v) {
        const int64_t u0 = u + (int64_t)(v - set) * t, w0 = u0 / share, w1 = (u0 + t - 1) / share;
        g.parts.first[v] = (int32_t)(kWaves * (w0 + s + v - set));
        g.parts.parts[v] = (int32_t)(w1 - w0 + 1);
        if (w1 > w0) whole = false;
      }
      const bool direct = whole && !x.shared && !x.split;
      if (direct) g.parts.first[0] = g.parts.first[1] = -1;
      g.slot = direct ? -1 : (int32_t)(blockIdx.x + s);
      // only offsets that are not ascending make more parts than there is room for
      if (g.slot >= 0 && kWaves * (g.slot + 1) > a.stream_units) g.x.cols = 0;
      atomicMax(n_seg, (int32_t)k + 1);
    });
  __syncthreads();
  // the list's end: the end of its last piece's stream, or of the share
  if (n_seg[0] < kSegments) return to;
  long long* end = n.sums;
  __syncthreads();
  walk([&](const Job&, int, int64_t u, int32_t t, int64_t s) {
    if (s - s_first == kSegments - 1) *end = min(to, u + t);
  });
  __syncthreads();
  return *end;
}


template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads, 2)
attend_stream_kernel(const AttendArgs a) {
  constexpr int PARTS = BF16_OUT ? 1 : 2;
  __shared__ __align__(16) uint16_t tile[kWaves][kStreamRows * (kStride + kVStride)];     // K rows, then V rows
  static_assert(sizeof(tile) >= kLengthsA + kLengthsB, "the lengths fit");
  __shared__ Segment seg[kSegments];
  __shared__ int32_t n_seg[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t layer = blockIdx.y;
  const int c = lane & 31, h = lane >> 5;
  const Lengths n = lengths_in(tile, reinterpret_cast<char*>(tile) + kLengthsA);
  uint16_t *kt = tile[wave], *vt = kt + kStreamRows * kStride;
  // rows by whole 16-lane groups: load i brings rows 4 i + (lane >> 4), dims 8 (lane & 15) .. + 7
  const int lr = lane >> 4, lc = 8 * (lane & 15);

  int64_t from = 0;
  for (;;) {
    const int64_t reached = list_segments(a, n, seg, n_seg, layer, from, tid);
    const int32_t ns = __builtin_amdgcn_readfirstlane(n_seg[0]);
    __syncthreads();                              // the lengths' memory becomes the tiles'

    // Two cursors run ahead of the tile that is computed, across the pieces: `where` finds rows (lane r the
    // r-th of the tile), one tile later they are loaded, one tile later used.
    struct Cursor {
      int32_t s, tile, tile1, nctx, c, p0, p1, seq;
      int64_t ck, pk;                             // element offsets of the memory rows and the pages
    } w, l;
    auto enter = [&](Cursor& u, int32_t s) {
      u.s = s;
      if (s >= ns) return;
      const Segment& g = seg[s];
      auto uni = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };
      u.tile = uni(g.tile0);
      u.tile1 = uni(g.tile1);
      u.c = uni(g.x.c);
      u.nctx = (u.c + kStreamRows - 1) / kStreamRows;
      u.p0 = uni(g.x.p0);
      u.p1 = uni(g.x.p1);
      u.seq = uni(g.x.seq);
      const int head = uni(g.set) * kWaves + wave;
      u.ck = (layer * a.n_groups + uni(g.x.grp)) * (int64_t)a.max_ctx * kRow + head * kDim;
      u.pk = ((layer * a.n_pages) << a.page_shift) * kRow + head * kDim;
    };
    auto step = [&](Cursor& u) {
      if (++u.tile >= u.tile1) enter(u, u.s + 1);
    };
    auto find = [&](const Cursor& u) -> int32_t {
      if (u.tile < u.nctx) return min(u.tile * kStreamRows + c, u.c - 1);
      const int32_t r = u.p0 + (u.tile - u.nctx) * kStreamRows + c;
      return u.p1 > u.p0 ? page_row(a, u.seq, min(r, u.p1 - 1)) : 0;
    };
    u32x4 pk[8], pv[8];
    auto load = [&](const Cursor& u, int32_t where) {
      const bool ctx = u.tile < u.nctx;
      const uint16_t* kb = ctx ? a.ctx_k + u.ck : a.k_pages + u.pk;
      const uint16_t* vb = ctx ? a.ctx_v + u.ck : a.v_pages + u.pk;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t off = (int64_t)__shfl(where, 4 * i + lr, 64) * kRow + lc;
        pk[i] = *reinterpret_cast<const u32x4*>(kb + off);
        pv[i] = *reinterpret_cast<const u32x4*>(vb + off);
      }
    };
    auto stage = [&](int32_t rows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        *reinterpret_cast<u32x4*>(kt + (4 * i + lr) * kStride + lc) = pk[i];
        if (rows < kStreamRows && 4 * i + lr >= rows) pv[i] = u32x4{0u, 0u, 0u, 0u};   // copies of the last row: weight 0
        *reinterpret_cast<u32x4*>(vt + (4 * i + lr) * kVStride + lc) = pv[i];
      }
    };
    enter(l, 0);
    w = l;
    int32_t where = 0;
    if (l.s < ns) {
      load(l, find(l));
      step(w);
      if (w.s < ns) where = find(w);
    }
    while (l.s < ns) {
      // one piece: columns, limits, tiles
      const int32_t s = l.s;
      const Job x = seg[s].x;
      const int head = seg[s].set * kWaves + wave;
      const int32_t slot = __builtin_amdgcn_readfirstlane(seg[s].slot);
      const Column y = column_of(a, x, layer, head, c);
      u32x4 qf[8];
      load_q(a, y, h, qf);
      // first local row (from p0) that the column does not see
      int32_t limit = 0;
      if (y.live && x.p1 > x.p0) {
        int32_t b = x.seq;
        if (x.shared) {                           // the token's sequence, searched from the group's first
          int32_t lo = b, hi = a.B - 1;
          while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (a.q_off[mid + 1] <= y.t) lo = mid + 1;
            else hi = mid;
          }
          b = lo;
        }
        limit = clampi(visible_rows(a, b, min(a.q_off[b + 1], a.n_q), y.t) - x.p0, 0, x.p1 - x.p0);
      }
      if (seg[s].first && wave == 0 && y.live && h == 0 && c % a.G == 0)
        describe(a, x, y, layer, seg[s].parts, 0, 1, kWaves, c);
      State st;
      clear(st);
      while (l.s == s) {
        const bool ctx = l.tile < l.nctx;
        const int32_t row0 = (ctx ? l.tile : l.tile - l.nctx) * kStreamRows;
        const int32_t rows = (ctx ? l.c : max(0, l.p1 - l.p0)) - row0;      // of this tile, or more
        const int32_t left = ctx ? rows : min(rows, limit - row0);
        stage(rows);
        l = w;
        if (l.s < ns) {
          load(l, where);
          step(w);
          if (w.s < ns) where = find(w);
        }
        attend32<PARTS, false>(kt, vt, qf, left, a.scale2, lane, st);     // rows bound the time: always masked
      }
      if (holds_nan(st)) {
        clear(st);
        Cursor u = l;
        enter(u, s);
        for (; u.tile < u.tile1; ++u.tile) {
          load(u, find(u));
          const bool ctx = u.tile < u.nctx;
          const int32_t row0 = (ctx ? u.tile : u.tile - u.nctx) * kStreamRows;
          const int32_t rows = (ctx ? u.c : max(0, u.p1 - u.p0)) - row0;
          stage(rows);
          attend32<PARTS, true>(kt, vt, qf, ctx ? rows : min(rows, limit - row0), a.scale2, lane, st);
        }
        if (l.s < ns) load(l, find(l));           // the next piece's first tile again
      }
      write_state<BF16_OUT>(a, st, y, layer, slot < 0 ? -1 : kWaves * slot + wave, lane);
    }
    from = reached;
    __syncthreads();
    if (ns < kSegments) return;                   // uniform
  }
}

// ------------------------------------------------------------------ more columns

struct Item {
  Job x;
  int32_t valid, nch, tile0, tile1;     // chunks of the job's tiles, this item's tiles
  int32_t head, col0, blocks;           // first column, column blocks (2 or 4)
  int32_t unit, first;                  // its first part (-1: writes the output), first chunk and head
  Parts parts;
};

// Fills `it` with this workgroup's item.  Items of a job: column blocks from the last (whose tokens see
// the most rows), chunks of rows, heads fastest (workgroups go to the 8 XCDs in turn: a head's rows
// stay in one L2).
__device__ __forceinline__ void find_item(const AttendArgs& a, const Lengths& n, Item& it, int64_t layer, int tid) {
  if (tid == 0) it.valid = 0;
  load_lengths(a, n, layer, tid);
  const int32_t nj = a.B + (a.grp_off ? a.n_groups : 0);
  const int32_t per = (nj + kThreads - 1) / kThreads, j0 = min(nj, tid * per), j1 = min(nj, j0 + per);
  long long work = 0, none = 0, all[2];
  for (int32_t j = j0; j < j1; ++j) {
    const Job x = job_of(a, n, j);
    if (x.cols > kCols) work += (long long)tiles_of(x, kTileRows) * ((x.cols + kWide - 1) / kWide) * kHeads;
  }
  scan2(n, work, none, all, tid);
  // tiles of a chunk: about as many items as aimed at, four tiles at least
  const int32_t aim = (int32_t)min((long long)1 << 25, max(4LL, (all[0] + a.tile_items - 1) / a.tile_items));
  auto chunks = [&](const Job& x) { return (tiles_of(x, kTileRows) + aim - 1) / aim; };
  long long items = 0, units = 0;
  for (int32_t j = j0; j < j1; ++j) {
    const Job x = job_of(a, n, j);
    if (x.cols <= kCols) continue;
    const int32_t nch = chunks(x);
    const long long k = (long long)nch * ((x.cols + kWide - 1) / kWide) * kHeads;
    items += k;
    if (x.shared || x.split || nch > 1) units += k;
  }
  const long long my_items = items, my_units = units;
  scan2(n, items, units, all, tid);
  const long long id = blockIdx.x;
  if (id >= items - my_items && id < items) {
    long long at = items - my_items, u = units - my_units;
    for (int32_t j = j0; j < j1; ++j) {
      const Job x = job_of(a, n, j);
      if (x.cols <= kCols) continue;
      const int32_t nch = chunks(x), ncb = (x.cols + kWide - 1) / kWide;
      const long long k = (long long)nch * ncb * kHeads;
      const bool parts = x.shared || x.split || nch > 1;
      if (id < at + k) {
        const int32_t i = (int32_t)(id - at), t = tiles_of(x, kTileRows);
        const int32_t chunk = i / kHeads % nch, xb = i / kHeads / nch, len = (t + nch - 1) / nch;
        it.x = x;
        it.nch = nch;
        it.head = i % kHeads;
        it.col0 = (ncb - 1 - xb) * kWide;
        it.blocks = x.cols - it.col0 <= 2 * kCols ? 2 : 4;
        it.tile0 = min(t, chunk * len);
        it.tile1 = min(t, it.tile0 + len);
        it.first = chunk == 0 && it.head == 0;
        it.unit = parts ? (int32_t)(a.stream_units + kWaves * (u + i)) : -1;
        for (int v = 0; v < kSets; ++v) {
          it.parts.first[v] = parts ? (int32_t)(a.stream_units + kWaves * (u + (long long)xb * nch * kHeads + v * kWaves)) : -1;
          it.parts.parts[v] = nch;
        }
        // only offsets that are not ascending make more parts than there is room for
        it.valid = !parts || a.stream_units + kWaves * (u + i + 1) <= a.max_units;
        break;
      }
      at += k;
      if (parts) u += k;
    }
  }
  __syncthreads();
}

// A stage of the tile kernel holds 64 K rows, then 64 V rows, 16 chunks of 16 bytes each, as the direct
// global -> LDS loads write them: lane l of load i brings chunk (l & 15) of row 4 i + (l >> 4).  The
// chunks of a row are permuted by the lanes' source addresses, so that fragment reads meet every bank
// once: chunk x of K row r lies at x ^ (r & 15) (16 rows, one chunk each), of V row r at
// x ^ 4 (r & 3) (4 rows, 4 chunks each).
constexpr int kStage = 2 * kTileRows * 16;        // u32x4

typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// This lane's pieces of K and V fragments in a stage: K rows 32 u + c, chunk 2 d + h is u32x4
// kx(u, d); the V rows of one transposed read start at element vx(u, m, half, d).
struct StageReads {
  int k0, v0;
  __device__ __forceinline__ explicit StageReads(int lane) {
    const int c = lane & 31, h = lane >> 5, i = lane & 15;
    k0 = c * 16 + (h ^ (c & 15));
    v0 = (kTileRows + 4 * h + (i >> 2)) * kDim + (4 * (i >> 2) + 2 * ((lane >> 4) & 1) + ((i >> 1) & 1)) * 8 + 4 * (i & 1);
  }
  __device__ __forceinline__ u32x4 k(const u32x4* stage, int u, int d) const { return stage[(k0 ^ (2 * d)) + 32 * 16 * u]; }
  __device__ __forceinline__ u32x4 v(const u32x4* stage, int u, int m, int d) const {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(stage) + (v0 ^ (32 * d)) + (32 * u + 16 * m) * kDim;
    return frag_of(lds_read_tr16(p), lds_read_tr16(p + 8 * kDim));
  }
};

// Rows 32 u .. 32 u + 31 of a stage into the state; a column sees the first `left` of them (whole: all do).
template <int PARTS, bool CAREFUL>
__device__ __forceinline__ void attend_stage(const u32x4* stage, const StageReads& at, int u, const u32x4* qf, bool whole,
                                             int32_t left, float scale2, int h, State& st) {
  f32x16 s = zeros16();
#pragma unroll
  for (int d = 0; d < 8; ++d) s = mfma32(at.k(stage, u, d), qf[d], s);
  u32x4 vf[2][4];               // on their way while the softmax runs
  if (!CAREFUL) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int d = 0; d < 4; ++d) vf[m][d] = at.v(stage, u, m, d);
  }
  if (!whole) {
    asm volatile("" ::: );      // a branch: most tiles are whole, and selects for all would cost what the exps do
    mask_rows(s, left, h);
  }
  raise_to(max16(s), scale2, st);
  const float neg_m = st.m == -__builtin_huge_valf() ? 0.f : -st.m;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    u32x4 ph, pl;
    weights<PARTS>(s, m, scale2, neg_m, ph, pl, st.l);
#pragma unroll
    for (int d = 0; d < 4; ++d)
      add_values<PARTS, CAREFUL>(CAREFUL ? at.v(stage, u, m, d) : vf[m][d], ph, pl, st.o[d]);
  }
}

template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads, 2)
attend_tile_kernel(const AttendArgs a) {
  constexpr int PARTS = BF16_OUT ? 1 : 2;
  // two arrays, so that the compiler sees which stage each access touches
  __shared__ u32x4 stage0[kStage], stage1[kStage];
  static_assert(sizeof(stage0) >= kLengthsA && sizeof(stage1) >= kLengthsB, "the lengths fit");
  __shared__ Item item;
  __shared__ int32_t s_most[kWaves];                 // local rows that a wave's columns see
  struct Half {
    float m[kCols], l[kCols];
    float o[kCols][kDim];
  };
  static_assert(sizeof(Half) <= sizeof(stage0), "a wave's state fits");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t layer = blockIdx.y;
  const int c = lane & 31, h = lane >> 5;
  const Lengths n = lengths_in(stage0, stage1);
  find_item(a, n, item, layer, tid);
  if (!item.valid) return;                           // uniform
  const Item& it = item;
  auto uni = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };
  const Job x = it.x;
  // two column blocks: two waves share a block's columns and take one half of each tile
  const int32_t blocks = uni(it.blocks), unit = uni(it.unit);
  const int32_t tile0 = uni(it.tile0), head = uni(it.head);
  int32_t tile1 = uni(it.tile1);
  const int cb = wave & (blocks - 1);
  const Column y = column_of(a, x, layer, head, it.col0 + cb * kCols + c);
  int32_t limit = 0;                                 // first local row (from p0) the column does not see
  if (y.live && x.p1 > x.p0) {
    const int32_t b = x.shared ? min(count_upto(n.off, a.B, y.t), a.B - 1) : x.seq;
    limit = clampi(visible_rows(a, b, n.off[b + 1], y.t) - x.p0, 0, x.p1 - x.p0);
  }
  int32_t most = limit, least = y.live ? limit : 0x7FFFFFFF;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    most = max(most, __shfl_xor(most, off, 64));
    least = min(least, __shfl_xor(least, off, 64));
  }
  most = uni(most);
  least = uni(least);
  u32x4 qf[8];
  load_q(a, y, h, qf);
  if (it.first && wave < blocks && y.live && h == 0 && c % a.G == 0)
    describe(a, x, y, layer, it.parts, it.unit < 0 ? 0 : cb, kWaves, kWaves * kHeads, c);
  if (lane == 0) s_most[wave] = most;
  __syncthreads();                                   // the lengths' memory becomes the tiles'

  const int32_t jc = uni(x.c), p0 = uni(x.p0), seq = uni(x.seq), nctx = (jc + kTileRows - 1) / kTileRows;
  int32_t wg_most = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) wg_most = max(wg_most, s_most[w]);
  wg_most = uni(wg_most);
  tile1 = min(tile1, nctx + (wg_most + kTileRows - 1) / kTileRows);

  // this wave's loads: rows 16 wave + 4 i + (lane >> 4) of K and of V
  constexpr int kPer = kTileRows / 4 / kWaves;
  const int lr = 4 * kPer * wave + (lane >> 4);
  const int64_t ctx_at = (layer * a.n_groups + uni(x.grp)) * (int64_t)a.max_ctx * kRow + head * kDim;
  const int64_t page_at = ((layer * a.n_pages) << a.page_shift) * kRow + head * kDim;
  int32_t where[kPer];
  auto find = [&](int32_t t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (t < nctx) where[i] = min(t * kTileRows + 4 * i + lr, jc - 1);
      else where[i] = page_row(a, seq, p0 + min((t - nctx) * kTileRows + 4 * i + lr, wg_most - 1));
    }
  };
  auto issue = [&](int32_t t, u32x4* stage) __attribute__((always_inline)) {
    const uint16_t* kb = t < nctx ? a.ctx_k + ctx_at : a.k_pages + page_at;
    const uint16_t* vb = t < nctx ? a.ctx_v + ctx_at : a.v_pages + page_at;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t row = (int64_t)where[i] * kRow;
      const int ck = (lane & 15) ^ ((4 * i + lr) & 15), cv = (lane & 15) ^ (4 * (lane >> 4));
      u32x4* to = stage + (kPer * wave + i) * 64;
      __builtin_amdgcn_global_load_lds((gptr_t)(kb + row + 8 * ck), (lptr_t)to, 16, 0, 0);
      __builtin_amdgcn_global_load_lds((gptr_t)(vb + row + 8 * cv), (lptr_t)(to + kTileRows * 16), 16, 0, 0);
    }
  };
  const StageReads at(lane);
  State st;
  clear(st);
  const int u0 = blocks == 2 ? wave >> 1 : 0, u1 = blocks == 2 ? u0 + 1 : 2;
  // rows of tile t, or more; rows of it that a column sees; rows that all the wave's columns see
  auto rows_of = [&](int32_t t) { return t < nctx ? jc - t * kTileRows : wg_most - (t - nctx) * kTileRows; };
  auto left_of = [&](int32_t t) { return t < nctx ? jc - t * kTileRows : limit - (t - nctx) * kTileRows; };
  auto all_of = [&](int32_t t) {
    return t < nctx ? jc - t * kTileRows : min(wg_most, least) - (t - nctx) * kTileRows;
  };
  // tile t is whole in its stage for every wave, and every wave is done with the stage before
  auto arrive = [&]() {
    __builtin_amdgcn_s_waitcnt(0);
    asm volatile("s_barrier" ::: "memory");
  };
  auto step = [&](int32_t t, const u32x4* stage, u32x4* other, auto two_halves) __attribute__((always_inline)) {
    arrive();
    if (t + 1 < tile1) issue(t + 1, other);
    if (t + 2 < tile1) find(t + 2);
    const int32_t all = all_of(t), left = left_of(t);
    if (two_halves) {
      attend_stage<PARTS, false>(stage, at, u0, qf, all >= 32 * u0 + 32, left - 32 * u0, a.scale2, h, st);
    } else {
      attend_stage<PARTS, false>(stage, at, 0, qf, all >= 32, left, a.scale2, h, st);
      attend_stage<PARTS, false>(stage, at, 1, qf, all >= 64, left - 32, a.scale2, h, st);
    }
  };
  auto run = [&](auto two_halves) __attribute__((always_inline)) {
    for (int32_t t = tile0; t < tile1; t += 2) {
      step(t, stage0, stage1, two_halves);
      if (t + 1 < tile1) step(t + 1, stage1, stage0, two_halves);
    }
  };
  if (tile0 < tile1) {
    find(tile0);
    issue(tile0, stage0);
    if (tile0 + 1 < tile1) find(tile0 + 1);
    if (blocks == 2) run(std::true_type());
    else run(std::false_type());
  }
  if (__syncthreads_or(holds_nan(st))) {
    clear(st);
    for (int32_t t = tile0; t < tile1; ++t) {
      find(t);
      issue(t, stage0);
      arrive();
#pragma unroll 1
      for (int u = u0; u < u1; ++u)
        attend_stage<PARTS, true>(stage0, at, u, qf, false, min(rows_of(t), left_of(t)) - 32 * u, a.scale2, h, st);
      __syncthreads();
    }
  }
  if (blocks == 2) {           // join the halves: waves 2 and 3 into waves 0 and 1
    __syncthreads();
    Half& z = *reinterpret_cast<Half*>(cb ? stage1 : stage0);
    if (wave >= 2) {
      const float l = halves_sum(st.l);
      if (h == 0) {
        z.m[c] = st.m;
        z.l[c] = l;
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(&z.o[c][32 * d + 8 * i + 4 * h]) =
              make_float4(st.o[d][4 * i], st.o[d][4 * i + 1], st.o[d][4 * i + 2], st.o[d][4 * i + 3]);
    }
    __syncthreads();
    if (wave >= 2) return;
    const float m = fmaxf(st.m, z.m[c]), base = m == -__builtin_huge_valf() ? 0.f : m;
    const float f = __builtin_amdgcn_exp2f(st.m - base), g = __builtin_amdgcn_exp2f(z.m[c] - base);
    st.m = m;
    st.l = st.l * f + (h == 0 ? z.l[c] * g : 0.f);
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[d][r] = st.o[d][r] * f + g * z.o[c][32 * d + 8 * (r >> 2) + 4 * h + (r & 3)];
  }
  write_state<BF16_OUT>(a, st, y, layer, unit < 0 ? -1 : unit + cb, lane);
}

// Joins the parts of a token's own rows and of its group's shared rows: four dims of one query head
// a thread, the parts in order with a running maximum.
template <bool BF16_OUT>
__global__ void __launch_bounds__(256)
attend_join_kernel(const AttendArgs a) {
  const int32_t t = blockIdx.x;
  const int64_t layer = blockIdx.z;
  if (t >= clampi(a.q_off[a.B], 0, a.n_q)) return;
  const int32_t i = blockIdx.y * 256 + threadIdx.x;
  const int32_t hq = i >> 5, d4 = 4 * (i & 31);
  if (hq >= a.Hq) return;
  const int4* desc = a.desc + (layer * a.n_q + t) * 4;
  const int32_t head = hq / a.G, hh = hq % a.G, set = head / kWaves;
  float m = -__builtin_huge_valf(), l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int which = 0, last = 0; which <= last; ++which) {
    const int4 d0 = desc[2 * which], d1 = desc[2 * which + 1];
    const int32_t first = set ? d0.z : d0.x, n = set ? d0.w : d0.y, col = d1.z + hh;
    if (which == 0) {
      if (first < 0) return;                // written by its item
      last = d1.w != 0;
    }
    const int32_t unit = first + (head % kWaves) * d1.x;
    // holds for every token of a sequence; offsets that are not ascending may leave a token without parts
    if (first < 0 || n < 1 || d1.x < 0 || d1.x > kWaves || d1.y < 0 || col < 0 || col >= a.unit_cols ||
        unit + (int64_t)(n - 1) * d1.y >= a.max_units)
      return;
    const int64_t at = (layer * a.max_units + unit) * a.unit_cols + col, step = (int64_t)d1.y * a.unit_cols;
    for (int32_t k0 = 0; k0 < n; k0 += 8) {
      float2 ml[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t p = at + min(k0 + u, n - 1) * step;
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
        if (k0 + u >= n) continue;
        const float w = __builtin_amdgcn_exp2f(ml[u].x - base);
        l += w * ml[u].y;
        o.x += w * v[u].x;
        o.y += w * v[u].y;
        o.z += w * v[u].z;
        o.w += w * v[u].w;
      }
      m = mn;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = ((layer * a.n_q + t) * a.Hq + hq) * kDim + d4;
  if (BF16_OUT)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(pack2_bf16(o.x * inv, o.y * inv), pack2_bf16(o.z * inv, o.w * inv));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

// Bounds for one layer.  Streamed pieces: one for each share and one more for each stream.  A tile job of
// n > 32 columns has 8 ceil(n / 128) <= n / 4 items a chunk (8 at 33), and cutting into chunks adds at
// most the number aimed at; parts come from all of them in groups, else only from jobs that are cut.
struct Sizes {
  int32_t stream_wgs, tile_items, items, unit_cols, stream_units, max_units;
  size_t desc, ml, acc, total;
};

Sizes sizes_of(int64_t L, int64_t B, int64_t n_groups, int64_t n_q, int64_t G) {
  Sizes z;
  const bool grouped = n_groups < B;
  const int64_t cols = n_q * G;
  auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  z.stream_wgs = (int32_t)(L < kStreamWgs ? kStreamWgs / L : 1);
  const int64_t jobs = least(B, n_q) + (grouped ? least(n_groups, n_q) : 0);
  z.stream_units = (int32_t)(kWaves * (z.stream_wgs + kSets * jobs));
  z.tile_items = z.items = 0;
  int64_t parts = 0;
  if (cols > kCols) {
    z.tile_items = (int32_t)(L < kTileItems ? kTileItems / L : 1);
    const int64_t items = z.tile_items + cols * (grouped ? 2 : 1) / 4;
    z.items = (int32_t)items;
    parts = grouped ? items : least(items, 2 * z.tile_items);
  }
  z.unit_cols = (int32_t)least(cols, kCols);
  z.max_units = (int32_t)(z.stream_units + kWaves * parts);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  z.desc = up((size_t)L * n_q * 4 * sizeof(int4));
  z.ml = up((size_t)L * z.max_units * z.unit_cols * sizeof(float2));
  z.acc = up((size_t)L * z.max_units * z.unit_cols * kDim * sizeof(float));
  z.total = z.desc + z.ml + z.acc;
  return z;
}

}  // namespace

size_t attend_workspace_bytes(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq) {
  return sizes_of(L, B, n_groups, n_q, Hq / kHeads).total;
}

template <bool BF16_OUT>
static void launch_attend_as(const AttendArgs& a, const Sizes& z, int32_t L, hipStream_t s) {
  if (z.items > 0)
    hipLaunchKernelGGL(attend_tile_kernel<BF16_OUT>, dim3((unsigned)z.items, (unsigned)L), dim3(kThreads), 0, s, a);
  hipLaunchKernelGGL(attend_stream_kernel<BF16_OUT>, dim3((unsigned)z.stream_wgs, (unsigned)L), dim3(kThreads), 0, s, a);
  hipLaunchKernelGGL(attend_join_kernel<BF16_OUT>,
                     dim3((unsigned)a.n_q, (unsigned)((a.Hq * 32 + 255) / 256), (unsigned)L), dim3(256), 0, s, a);
}

hipError_t launch_attend(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* q,
                         const int32_t* q_off, const int32_t* grp_off, const uint16_t* ctx_k, const uint16_t* ctx_v,
                         const int32_t* ctx_len, int32_t max_ctx, const uint16_t* k_pages, const uint16_t* v_pages,
                         int32_t n_pages, int32_t page_shift, const int32_t* page_table, int32_t max_pages,
                         const int32_t* kv_len, const int32_t* pre_len, float scale, bool bf16_out, void* out,
                         void* ws, hipStream_t s) {
  const Sizes z = sizes_of(L, B, n_groups, n_q, Hq / kHeads);
  char* w = static_cast<char*>(ws);
  const AttendArgs a = {B, n_groups, n_q, Hq, Hq / kHeads, max_ctx, n_pages, page_shift, max_pages, q, q_off, grp_off,
                        ctx_k, ctx_v, ctx_len, k_pages, v_pages, page_table, kv_len, pre_len,
                        scale * 1.4426950408889634f, out, z.stream_wgs, z.tile_items, z.unit_cols, z.stream_units,
                        z.max_units, reinterpret_cast<int4*>(w), reinterpret_cast<float2*>(w + z.desc),
                        reinterpret_cast<float*>(w + z.desc + z.ml)};
  if (bf16_out) launch_attend_as<true>(a, z, L, s);
  else launch_attend_as<false>(a, z, L, s);
  return hipGetLastError();
}

}  // namespace msa
