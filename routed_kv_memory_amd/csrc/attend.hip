// attend.hip -- attention of ragged new tokens over [memory context ; paged local rows], the
// context and the first local pages shared by the sequences of a group.
//
// For every layer, token i of sequence b (n_b new tokens) in group g sees the group's memory rows
// 0 .. ctx_len[g]) and its local rows 0 .. kv_len[b] - n_b + i; query head hq reads KV head
// hq / (Hq / 8); the output is the softmax-weighted sum of the visible V rows.
//
// The work is a list of jobs: a job is a set of columns (token, query head of one KV head; the G
// heads of a token side by side) over a row space [c memory rows ; local rows p0 .. p1).  A group of
// several sequences makes one job of all its tokens over the shared rows and one job for each
// sequence over its own rows; a sequence alone in its group makes one job over everything.  Every
// column has one limit: the rows of the job's space below it are visible.  Lengths are on the
// device, so each workgroup forms the list itself (a few loads and two scans over the jobs, in LDS)
// and takes the item that has its number; the host only bounds the number of items.
//
// A wave always holds 32 columns.  On the matrix cores (v_mfma_f32_32x32x16_bf16), per 32 rows:
// S^T = K . Q^T with K as the A operand and the columns as the B operand (registers), so lane l has
// column l & 31 and the rows 8 i + 4 (l >> 5) + 0..3; the softmax needs one exchange between the
// two halves of the wave.  For O^T += V^T . P^T the MFMA's k axis is taken in the order in which the
// scores already lie in the lanes, and V^T comes from the row-major tile by transposed LDS reads.
//
// Jobs of up to 128 columns are bound by HBM: each wave streams its own rows through a tile of its
// own in LDS, without barriers; the 8 waves of a workgroup take 8 (head, column block) pairs of the
// same rows, so a row's 2 KiB are read together.  Jobs of more columns are bound by the matrix cores:
// 8 waves of one head share each tile of 64 rows, 256 columns a workgroup.  Row ranges are cut into
// chunks so that a call makes about kItems items; parts are joined by a second kernel, and a job
// that is whole in one chunk writes its output itself.
#include "msa_device.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kCols = 32;                 // columns of a wave
constexpr int kNarrow = 4 * kCols;        // most columns of a job that is streamed
constexpr int kWide = kWaves * kCols;     // columns of a workgroup otherwise
constexpr int kStreamRows = 32;           // rows of a streamed tile
constexpr int kTileRows = 64;             // rows of a shared tile
constexpr int kStride = kDim + 8;         // bf16 per staged row
constexpr int kMaxSeqs = 2048;            // MSA_MAX_SEQS
constexpr int kStreamItems = 512;         // items a call aims at, by kind
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
  int32_t stream_items, tile_items;       // items aimed at in one layer
  int32_t unit_cols, max_units;           // columns of a part in the workspace, parts of one layer
  int4* desc;                             // [L][n_q][2]: where a token's parts are (own rows, shared rows)
  float2* ml;                             // [L][max_units][unit_cols]: maximum (log2 units) and sum
  float* acc;                             // [L][max_units][unit_cols][128]
};

struct Job {
  int32_t t0, cols;        // first packed token, columns
  int32_t seq, grp;        // whose page table, whose memory rows
  int32_t c, p0, p1;       // memory rows, local rows [p0, p1)
  bool shared, split;      // the group's shared rows; own rows next to a shared job
};

// The lengths of one layer, clamped, in LDS.
struct Lengths {
  int32_t off[kMaxSeqs + 1], len[kMaxSeqs];
  int32_t grp[kMaxSeqs + 1], clen[kMaxSeqs], pre[kMaxSeqs];
};

struct Item {
  Job job;
  int32_t wide, nch, chunk;     // chunks of the job, this item's
  int32_t r0, r1;               // its rows
  int32_t col0, ncb, head;      // first column; streamed: column blocks, first head
  int32_t unit;                 // first of its 8 parts, -1: writes the output itself
  int32_t unit_k0;              // the same of chunk 0 and head 0
};

union Shared {
  struct {
    Lengths n;
    int32_t sums[kWaves][3];
    int64_t work[kWaves][2];
    Item item;
  } plan;
  uint16_t stream[kWaves][2][kStreamRows * kStride];
  uint16_t tile[2][2][kTileRows * kStride];
};

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

// Jobs 0 .. n_groups) are the groups' shared rows (none when every sequence is its own group), then
// one for each sequence.
__device__ __forceinline__ Job job_of(const AttendArgs& a, const Lengths& n, int32_t j) {
  const bool grouped = a.grp_off != nullptr;
  const int32_t ng = grouped ? a.n_groups : 0;
  Job x;
  x.cols = 0;
  x.split = false;
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
  x.p1 = n.len[b];
  if (!grouped) {
    x.grp = b;
    x.c = n.clen[b];
    x.p0 = 0;
    return x;
  }
  const int32_t g = count_upto(n.grp, a.n_groups, b);
  const bool in = g < a.n_groups && n.grp[g] <= b;   // a sequence outside all groups has no memory rows
  x.grp = in ? g : 0;
  const int32_t c = in ? n.clen[g] : 0;
  if (in && n.grp[g + 1] - n.grp[g] > 1) {
    x.c = 0;
    x.p0 = n.pre[g];
    x.split = c + x.p0 > 0;
  } else {
    x.c = c;
    x.p0 = 0;
  }
  return x;
}

__device__ __forceinline__ int32_t job_rows(const Job& x) { return x.c + max(0, x.p1 - x.p0); }
__device__ __forceinline__ int32_t col_blocks(int32_t cols) { return cols <= kCols ? 1 : (cols <= 2 * kCols ? 2 : 4); }
__device__ __forceinline__ int32_t tiles_of(int32_t rows, int32_t t) { return rows > 0 ? (rows + t - 1) / t : 1; }

__device__ __forceinline__ int32_t wave_scan_incl(int32_t v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor((long long)v, off, 64);
  return v;
}

// Fills sh.plan.item with this workgroup's item; false when there is none.  Ends on a barrier.
__device__ bool make_plan(const AttendArgs& a, Shared& sh, int64_t layer, int tid) {
  Lengths& n = sh.plan.n;
  const bool grouped = a.grp_off != nullptr;
  const int32_t cap = a.max_pages << a.page_shift;
  const int lane = tid & 63, wave = tid >> 6;
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
  if (tid == 0) sh.plan.item.wide = -1;
  __syncthreads();
  const int32_t nj = a.B + (grouped ? a.n_groups : 0);
  const int32_t per = (nj + kThreads - 1) / kThreads;
  const int32_t j0 = min(nj, tid * per), j1 = min(nj, j0 + per);
  // work of each kind: streamed tiles x column blocks, shared tiles x heads x column blocks
  int64_t un = 0, uw = 0;
  for (int32_t j = j0; j < j1; ++j) {
    const Job x = job_of(a, n, j);
    if (x.cols == 0) continue;
    if (x.cols <= kNarrow) un += (int64_t)tiles_of(job_rows(x), kStreamRows) * col_blocks(x.cols);
    else uw += (int64_t)tiles_of(job_rows(x), kTileRows) * ((x.cols + kWide - 1) / kWide) * kHeads;
  }
  un = wave_sum64(un);
  uw = wave_sum64(uw);
  if (lane == 0) {
    sh.plan.work[wave][0] = un;
    sh.plan.work[wave][1] = uw;
  }
  __syncthreads();
  int64_t tn = 0, tw = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    tn += sh.plan.work[w][0];
    tw += sh.plan.work[w][1];
  }
  // tiles of a chunk: about as many items as aimed at, by kind (a chunk's rows stay within 2^30)
  const int64_t most = ((int64_t)1 << 30) / kStreamRows;
  const int32_t cn = (int32_t)min(most, max((int64_t)1, (tn + a.stream_items - 1) / a.stream_items));
  const int32_t cw = (int32_t)min(most / 2, max((int64_t)4, (tw + a.tile_items - 1) / max(1, a.tile_items)));
  // items and parts of this thread's jobs, then where they start
  int32_t in = 0, iw = 0, iu = 0;
  auto items_of = [&](const Job& x, int32_t& nch) {
    if (x.cols <= kNarrow) {
      nch = (tiles_of(job_rows(x), kStreamRows) + cn - 1) / cn;
      return nch * col_blocks(x.cols);
    }
    nch = (tiles_of(job_rows(x), kTileRows) + cw - 1) / cw;
    return nch * ((x.cols + kWide - 1) / kWide) * kHeads;
  };
  for (int32_t j = j0; j < j1; ++j) {
    const Job x = job_of(a, n, j);
    if (x.cols == 0) continue;
    int32_t nch;
    const int32_t k = items_of(x, nch);
    (x.cols <= kNarrow ? in : iw) += k;
    if (x.shared || x.split || nch > 1) iu += k;
  }
  const int32_t en = wave_scan_incl(in, lane), ew = wave_scan_incl(iw, lane), eu = wave_scan_incl(iu, lane);
  if (lane == 63) {
    sh.plan.sums[wave][0] = en;
    sh.plan.sums[wave][1] = ew;
    sh.plan.sums[wave][2] = eu;
  }
  __syncthreads();
  int32_t bn = en - in, bw = ew - iw, bu = eu - iu, all_w = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) {
      bn += sh.plan.sums[w][0];
      bw += sh.plan.sums[w][1];
      bu += sh.plan.sums[w][2];
    }
    all_w += sh.plan.sums[w][1];
  }
  bn += all_w;                              // the long shared-tile items start first
  const int32_t id = blockIdx.x;
  if ((id >= bw && id < bw + iw) || (id >= bn && id < bn + in)) {
    for (int32_t j = j0; j < j1; ++j) {
      const Job x = job_of(a, n, j);
      if (x.cols == 0) continue;
      int32_t nch;
      const int32_t k = items_of(x, nch);
      const bool parts = x.shared || x.split || nch > 1;
      const bool wide = x.cols > kNarrow;
      int32_t& base = wide ? bw : bn;
      if (id >= base && id < base + k) {
        Item& it = sh.plan.item;
        const int32_t i = id - base, rows = job_rows(x);
        it.job = x;
        it.wide = wide;
        it.nch = nch;
        int32_t len;
        if (wide) {
          // heads fastest (workgroups go to the 8 XCDs in turn: a head's rows stay in one L2); the
          // last tokens' columns, which see the most rows, first
          const int32_t ncw = (x.cols + kWide - 1) / kWide;
          it.head = i % kHeads;
          it.chunk = (i / kHeads) % nch;
          const int32_t cb = ncw - 1 - i / kHeads / nch;
          it.col0 = cb * kWide;
          it.ncb = kWaves;
          it.unit_k0 = 8 * (bu + (ncw - 1 - cb) * nch * kHeads);
          len = cw * kTileRows;
        } else {
          it.ncb = col_blocks(x.cols);
          it.chunk = i / it.ncb;
          it.head = (i % it.ncb) * (kWaves / it.ncb);
          it.col0 = 0;
          it.unit_k0 = 8 * bu;
          len = cn * kStreamRows;
        }
        it.unit = parts ? 8 * (bu + i) : -1;
        if (parts && it.unit + 8 > a.max_units) it.wide = -1;     // only for offsets that are not ascending
        it.r0 = it.chunk * len;
        it.r1 = min(rows, it.r0 + len);
      }
      base += k;
      if (parts) bu += k;
    }
  }
  __syncthreads();
  return sh.plan.item.wide >= 0;
}

// Where row `r` of the job's space lies: a row of the page pool (>= 0) or ~(memory row).
__device__ __forceinline__ int32_t row_at(const AttendArgs& a, const Job& x, int32_t r) {
  if (r < x.c) return ~r;
  const int32_t lr = x.p0 + r - x.c;
  const int32_t page = clampi(a.page_table[(int64_t)x.seq * a.max_pages + (lr >> a.page_shift)], 0, a.n_pages - 1);
  return (page << a.page_shift) + (lr & ((1 << a.page_shift) - 1));
}

struct RowBases {
  const uint16_t *ck, *cv, *pk, *pv;
};

__device__ __forceinline__ RowBases row_bases(const AttendArgs& a, const Job& x, int64_t layer, int head) {
  const int64_t ctx = (layer * a.n_groups + x.grp) * (int64_t)a.max_ctx * kRow + head * kDim;
  const int64_t pages = ((layer * a.n_pages) << a.page_shift) * kRow + head * kDim;
  return RowBases{a.ctx_k + ctx, a.ctx_v + ctx, a.k_pages + pages, a.v_pages + pages};
}

// A wave's running state: lane l holds column l & 31; dims 32 d + 8 (r >> 2) + 4 (l >> 5) + (r & 3) of it.
struct State {
  float m, l;
  f32x16 o[4];
};

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

// Rows row0 .. row0 + 31 (tiles kt, vt in LDS) into the state of the wave's 32 columns.  `whole`
// (uniform): every column sees all of them; otherwise the rows from `limit` on are masked.
// PARTS: 2 puts the probabilities into the second product as bf16 high part + bf16 residual, 1 as
// one bf16 value, whose rounding (2^-9 of each weight) is the size of a bf16 output's own; the sum
// is then taken of the rounded values, so the weights still add up to one.
template <int PARTS>
__device__ __forceinline__ void attend32(const uint16_t* kt, const uint16_t* vt, const u32x4* qf, int32_t row0,
                                         int32_t limit, bool whole, float scale2, int lane, State& st) {
  const int c = lane & 31, h = lane >> 5;
  f32x16 s = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < 8; ++d)
    s = mfma32(*reinterpret_cast<const u32x4*>(kt + c * kStride + 16 * d + 8 * h), qf[d], s);
  const float ninf = -__builtin_huge_valf();
  if (!whole) {
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = row0 + 8 * (r >> 2) + 4 * h + (r & 3) < limit ? s[r] : ninf;
  }
  float mt = s[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) mt = fmaxf(mt, s[r]);
  mt = halves_max(mt) * scale2;
  // the reference maximum is raised only when a tile passes it by more than 2^8: most skip the rescale
  const bool raise = mt > st.m + 8.f;
  if (__ballot(raise)) {
    const float mn = raise ? mt : st.m;
    const float alpha = st.m == ninf ? 0.f : __builtin_amdgcn_exp2f(st.m - mn);
    st.m = raise ? mt : st.m;
    if (raise) {
      st.l *= alpha;
#pragma unroll
      for (int d = 0; d < 4; ++d) st.o[d] *= alpha;
    }
  }
  const float neg_m = st.m == ninf ? 0.f : -st.m;
#pragma unroll
  for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale2, neg_m));
  u32x4 ph[2], pl[2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p0 = s[8 * m + 2 * e], p1 = s[8 * m + 2 * e + 1];
      const uint32_t w = pack2_bf16(p0, p1);
      ph[m][e] = w;
      if (PARTS == 2) {
        pl[m][e] = pack2_bf16(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xFFFF0000u));
        st.l += p0 + p1;
      } else {
        st.l += __uint_as_float(w << 16) + __uint_as_float(w & 0xFFFF0000u);
      }
    }
  // k slot 8 h + e of product m holds row 16 m + 4 h + e (e < 4) or 16 m + 8 + 4 h + e - 4; a 16-lane
  // group reads 16 dims of 4 rows transposed
  const int i = lane & 15;
  const uint16_t* vsrc = vt + (4 * h + (i >> 2)) * kStride + 16 * ((lane >> 4) & 1) + 4 * (i & 3);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint2 v0 = lds_read_tr16(vsrc + 16 * m * kStride + 32 * d);
      const uint2 v1 = lds_read_tr16(vsrc + (16 * m + 8) * kStride + 32 * d);
      u32x4 vf = {v0.x, v0.y, v1.x, v1.y};
      if (!whole) {
        // a masked row's weight is 0, but 0 * inf is NaN: entries that are not finite are taken out of
        // the product and their kind is added where a weight above 0 meets one
        u32x4 bad;
#pragma unroll
        for (int e = 0; e < 4; ++e) bad[e] = not_finite(vf[e]);
        if (__ballot((bad[0] | bad[1] | bad[2] | bad[3]) != 0)) {
          const u32x4 raw = vf;
          vf &= ~bad;
#pragma unroll
          for (int kind = 0; kind < 3; ++kind) {
            u32x4 one;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = raw[e] & 0xFFFFu, hi = raw[e] >> 16;
              auto is = [&](uint32_t x) {
                return kind == 0 ? x == 0x7F80u : (kind == 1 ? x == 0xFF80u : (x & 0x7FFFu) > 0x7F80u);
              };
              one[e] = (is(lo) ? 0x3F80u : 0u) | (is(hi) ? 0x3F800000u : 0u);
            }
            f32x16 t = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            t = mfma32(one, ph[m], t);
            const float add = kind == 0 ? -ninf : (kind == 1 ? ninf : __builtin_nanf(""));
#pragma unroll
            for (int r = 0; r < 16; ++r) st.o[d][r] += t[r] > 0.f ? add : 0.f;
          }
        }
      }
      st.o[d] = mfma32(vf, ph[m], st.o[d]);
      if (PARTS == 2) st.o[d] = mfma32(vf, pl[m], st.o[d]);
    }
}

template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads)
attend_kernel(const AttendArgs a) {
  constexpr int PARTS = BF16_OUT ? 1 : 2;
  __shared__ __align__(16) Shared sh;
  __shared__ int32_t s_end[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t layer = blockIdx.y;
  if (!make_plan(a, sh, layer, tid)) return;         // uniform
  const Item it = sh.plan.item;
  const Job x = it.job;
  const int c = lane & 31, h = lane >> 5;

  // this wave's head and columns, each column's limit
  const int cb = it.wide ? wave : wave % it.ncb;
  const int head = it.wide ? it.head : it.head + wave / it.ncb;
  const int32_t col = it.col0 + cb * kCols + c;
  const bool live = col < x.cols;
  const int32_t t = x.t0 + (live ? col / a.G : 0);
  int32_t limit = 0;
  if (live) {
    const Lengths& n = sh.plan.n;
    const int32_t b = x.shared ? min(count_upto(n.off, a.B, t), a.B - 1) : x.seq;
    // the token's visible local rows are 0 .. lim)
    const int32_t lim = n.len[b] == 0 ? 0 : a.kv_len[b] - (n.off[b + 1] - t) + 1;
    limit = x.c + clampi(lim - x.p0, 0, max(0, x.p1 - x.p0));
  }
  // rows this wave needs, rows all its columns see
  int32_t most = limit, least = live ? limit : 0x7FFFFFFF;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    most = max(most, __shfl_xor(most, off, 64));
    least = min(least, __shfl_xor(least, off, 64));
  }
  const int32_t end = __builtin_amdgcn_readfirstlane(min(it.r1, most));
  const int32_t all = __builtin_amdgcn_readfirstlane(least);
  const int64_t q_row = (layer * a.n_q + t) * a.Hq + head * a.G + (live ? col % a.G : 0);
  u32x4 qf[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    qf[d] = u32x4{0u, 0u, 0u, 0u};
    if (live) qf[d] = *reinterpret_cast<const u32x4*>(a.q + q_row * kDim + 16 * d + 8 * h);
  }
  // where the parts of this item's tokens are, from the item of chunk 0 and the first head
  if (it.chunk == 0 && (it.wide ? it.head == 0 : head == 0) && live && h == 0 && col % a.G == 0) {
    int4 d;
    d.x = it.unit < 0 ? -1 : it.unit_k0 + cb;
    d.y = it.nch;
    d.z = it.ncb | (c << 8);
    d.w = x.split;
    a.desc[(layer * a.n_q + t) * 2 + (x.shared ? 1 : 0)] = d;
  }
  if (lane == 0) s_end[wave] = end;
  __syncthreads();                                   // the plan's memory becomes the tiles'

  State st;
  st.m = -__builtin_huge_valf();
  st.l = 0.f;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) st.o[d][r] = 0.f;

  if (!it.wide) {
    // rows of whole 16-lane groups: load i brings rows 4 i + (lane >> 4), dims 8 (lane & 15) .. + 7
    const RowBases rb = row_bases(a, x, layer, head);
    uint16_t *kt = sh.stream[wave][0], *vt = sh.stream[wave][1];
    const int lr = lane >> 4, lc = 8 * (lane & 15);
    u32x4 pk[8], pv[8];
    auto load = [&](int32_t where, int32_t row0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t at = __shfl(where, 4 * i + lr, 64);
        const int64_t off = (int64_t)(at < 0 ? ~at : at) * kRow + lc;
        pk[i] = *reinterpret_cast<const u32x4*>((at < 0 ? rb.ck : rb.pk) + off);
        pv[i] = *reinterpret_cast<const u32x4*>((at < 0 ? rb.cv : rb.pv) + off);
      }
    };
    if (it.r0 < end) {
      int32_t where = row_at(a, x, min(it.r0 + c, end - 1));
      load(where, it.r0);
      where = row_at(a, x, min(it.r0 + kStreamRows + c, end - 1));
      for (int32_t row0 = it.r0; row0 < end; row0 += kStreamRows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          *reinterpret_cast<u32x4*>(kt + (4 * i + lr) * kStride + lc) = pk[i];
          // rows past the end (copies of the last one) hold zeros in V: their weight is 0
          *reinterpret_cast<u32x4*>(vt + (4 * i + lr) * kStride + lc) =
              row0 + 4 * i + lr < end ? pv[i] : u32x4{0u, 0u, 0u, 0u};
        }
        if (row0 + kStreamRows < end) {
          load(where, row0 + kStreamRows);
          where = row_at(a, x, min(row0 + 2 * kStreamRows + c, end - 1));
        }
        attend32<PARTS>(kt, vt, qf, row0, min(limit, end), row0 + kStreamRows <= min(all, end), a.scale2, lane, st);
      }
    }
  } else {
    const RowBases rb = row_bases(a, x, layer, it.head);
    int32_t wg_end = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) wg_end = max(wg_end, s_end[w]);
    const int lr = tid >> 4, lc = 8 * (tid & 15);
    u32x4 pk[2], pv[2];
    int32_t where[2];
    auto find = [&](int32_t row0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) where[i] = row_at(a, x, min(row0 + 32 * i + lr, wg_end - 1));
    };
    auto load = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t at = where[i];
        const int64_t off = (int64_t)(at < 0 ? ~at : at) * kRow + lc;
        pk[i] = *reinterpret_cast<const u32x4*>((at < 0 ? rb.ck : rb.pk) + off);
        pv[i] = *reinterpret_cast<const u32x4*>((at < 0 ? rb.cv : rb.pv) + off);
      }
    };
    auto store = [&](int buf, int32_t row0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<u32x4*>(sh.tile[buf][0] + (32 * i + lr) * kStride + lc) = pk[i];
        *reinterpret_cast<u32x4*>(sh.tile[buf][1] + (32 * i + lr) * kStride + lc) =
            row0 + 32 * i + lr < wg_end ? pv[i] : u32x4{0u, 0u, 0u, 0u};
      }
    };
    if (it.r0 < wg_end) {
      find(it.r0);
      load();
      store(0, it.r0);
      find(it.r0 + kTileRows);
      int buf = 0;
      for (int32_t row0 = it.r0; row0 < wg_end; row0 += kTileRows, buf ^= 1) {
        __syncthreads();       // the tile is in buf; every reader of buf ^ 1 (the tile before) is done
        const bool more = row0 + kTileRows < wg_end;
        if (more) {
          load();
          find(row0 + 2 * kTileRows);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int32_t r = row0 + 32 * u;
          if (r < end)
            attend32<PARTS>(sh.tile[buf][0] + 32 * u * kStride, sh.tile[buf][1] + 32 * u * kStride, qf, r, min(limit, end),
                            r + 32 <= min(all, end), a.scale2, lane, st);
        }
        if (more) store(buf ^ 1, row0 + kTileRows);
      }
    }
  }

  st.l = halves_sum(st.l);
  if (!live) return;
  if (it.unit < 0) {
    const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = q_row * kDim + 32 * d + 8 * i + 4 * h;
        const float v0 = st.o[d][4 * i] * inv, v1 = st.o[d][4 * i + 1] * inv, v2 = st.o[d][4 * i + 2] * inv,
                    v3 = st.o[d][4 * i + 3] * inv;
        if (BF16_OUT)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack2_bf16(v0, v1), pack2_bf16(v2, v3));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v0, v1, v2, v3);
      }
  } else {
    const int64_t part = (layer * a.max_units + it.unit + wave) * a.unit_cols + c;
    if (h == 0) a.ml[part] = make_float2(st.m, st.l);
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(a.acc + part * kDim + 32 * d + 8 * i + 4 * h) =
            make_float4(st.o[d][4 * i], st.o[d][4 * i + 1], st.o[d][4 * i + 2], st.o[d][4 * i + 3]);
  }
}

// Joins the parts of a token's own rows and of its group's shared rows: four dims of one query head
// a thread, the parts in order with a running maximum.
template <bool BF16_OUT>
__global__ void __launch_bounds__(256)
attend_join_kernel(const AttendArgs a) {
  const int32_t t = blockIdx.x;
  const int64_t layer = blockIdx.z;
  const int32_t seqs_end = clampi(a.q_off[a.B], 0, a.n_q);
  if (t >= seqs_end) return;
  const int32_t i = blockIdx.y * 256 + threadIdx.x;
  const int32_t hq = i >> 5, d4 = 4 * (i & 31);
  if (hq >= a.Hq) return;
  const int4* desc = a.desc + (layer * a.n_q + t) * 2;
  const int4 own = desc[0];
  if (own.x < 0) return;                    // written by its item
  const int32_t head = hq / a.G, hh = hq % a.G;
  float m = -__builtin_huge_valf(), l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int which = 0; which < (own.w ? 2 : 1); ++which) {
    const int4 d = which ? desc[1] : own;
    const int32_t hs = d.z & 255, nch = d.y;
    // holds for every token of a sequence; offsets that are not ascending may leave a token without parts
    if (d.x < 0 || nch < 1 || hs > kWaves || (d.z >> 8) + hh >= a.unit_cols ||
        d.x + (int64_t)hs * head + (int64_t)8 * hs * (nch - 1) >= a.max_units)
      return;
    const int64_t first = (layer * a.max_units + d.x + hs * head) * a.unit_cols + (d.z >> 8) + hh;
    const int64_t step = (int64_t)8 * hs * a.unit_cols;
    for (int32_t k0 = 0; k0 < nch; k0 += 8) {
      float2 ml[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t p = first + min(k0 + u, nch - 1) * step;
        ml[u] = a.ml[p];
        v[u] = *reinterpret_cast<const float4*>(a.acc + p * kDim + d4);
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < 8; ++u) mn = fmaxf(mn, ml[u].x);
      m = m == -__builtin_huge_valf() ? m : m - mn;     // no row so far: a factor of 0
      const float base = mn == -__builtin_huge_valf() ? 0.f : mn;
      const float s = __builtin_amdgcn_exp2f(m);
      l *= s;
      o.x *= s;
      o.y *= s;
      o.z *= s;
      o.w *= s;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (k0 + u >= nch) continue;
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

// Bounds on one layer's items and parts.  A streamed job of n columns has col_blocks(n) <= max(1, n / 16)
// items a chunk, a wide one 8 ceil(n / 256) <= n / 16; chunks are sized so that cutting adds at
// most the number aimed at.  Jobs with parts: all of them in groups, else only those that are cut.
struct Sizes {
  int32_t stream_items, tile_items, items, unit_cols, max_units;
  size_t desc, ml, acc, total;
};

Sizes sizes_of(int64_t L, int64_t B, int64_t n_groups, int64_t n_q, int64_t G) {
  Sizes z;
  const bool grouped = n_groups < B;
  const int64_t cols = n_q * G;
  z.stream_items = (int32_t)((kStreamItems + L - 1) / L);
  z.tile_items = cols > kNarrow ? (int32_t)((kTileItems + L - 1) / L) : 0;
  const int64_t jobs = (B < n_q ? B : n_q) + (grouped ? (n_groups < n_q ? n_groups : n_q) : 0);
  const int64_t aimed = z.stream_items + z.tile_items;
  const int64_t items = aimed + jobs + cols * (grouped ? 2 : 1) / 16;
  z.items = (int32_t)items;
  z.unit_cols = (int32_t)(cols < kCols ? cols : kCols);
  z.max_units = (int32_t)(8 * (grouped || items < 2 * aimed ? items : 2 * aimed));
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  z.desc = up((size_t)L * n_q * 2 * sizeof(int4));
  z.ml = up((size_t)L * z.max_units * z.unit_cols * sizeof(float2));
  z.acc = up((size_t)L * z.max_units * z.unit_cols * kDim * sizeof(float));
  z.total = z.desc + z.ml + z.acc;
  return z;
}

}  // namespace

size_t attend_workspace_bytes(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq) {
  return sizes_of(L, B, n_groups, n_q, Hq / kHeads).total;
}

hipError_t launch_attend(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* q,
                         const int32_t* q_off, const int32_t* grp_off, const uint16_t* ctx_k, const uint16_t* ctx_v,
                         const int32_t* ctx_len, int32_t max_ctx, const uint16_t* k_pages, const uint16_t* v_pages,
                         int32_t n_pages, int32_t page_shift, const int32_t* page_table, int32_t max_pages,
                         const int32_t* kv_len, const int32_t* pre_len, float scale, bool bf16_out, void* out,
                         void* ws, hipStream_t s) {
  const Sizes z = sizes_of(L, B, n_groups, n_q, Hq / kHeads);
  char* w = static_cast<char*>(ws);
  AttendArgs a = {B, n_groups, n_q, Hq, Hq / kHeads, max_ctx, n_pages, page_shift, max_pages, q, q_off, grp_off, ctx_k,
                  ctx_v, ctx_len, k_pages, v_pages, page_table, kv_len, pre_len, scale * 1.4426950408889634f, out,
                  z.stream_items, z.tile_items, z.unit_cols, z.max_units, reinterpret_cast<int4*>(w),
                  reinterpret_cast<float2*>(w + z.desc), reinterpret_cast<float*>(w + z.desc + z.ml)};
  const dim3 grid((unsigned)z.items, (unsigned)L), join((unsigned)n_q, (unsigned)((Hq * 32 + 255) / 256), (unsigned)L);
  if (bf16_out) {
    hipLaunchKernelGGL(attend_kernel<true>, grid, dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(attend_join_kernel<true>, join, dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL(attend_kernel<false>, grid, dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(attend_join_kernel<false>, join, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace msa
