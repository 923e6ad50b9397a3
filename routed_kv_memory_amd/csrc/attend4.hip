// attend4.hip -- attention of ragged new tokens over [memory context ; paged local rows held in 4 bits].
//
// What attend.hip computes, over local rows in the format of cache4.hpp; the memory rows are bf16.  A code stands
// for an exact bf16 value, so the rows are turned into those on the way to the matrix cores, and the arithmetic is that
// of the attention over rows in bf16.  (Scaled products of the codes themselves would need q in 8 bits: in two parts
// of them a score is off by up to 2^-13.6 of its sum of magnitudes, 2^-20 here.)
//
// - Jobs of up to 16 columns: a wave streams rows, of the memory 16 a tile, of the pages 64, which are as many bytes
//   and go through the same registers (tiles of 32 and 128: 763 us where these take 248, they spill).  K codes
//   are loaded as the first product's A operand takes them (lane l: 32 dims, a block with its scale, of row l & 15) and
//   turned into bf16 in registers; V's codes wait in the wave's LDS tile, so that their registers take the next
//   tile's, and are turned into bf16 there 32 rows at a time.  Bound: HBM.  One token over 36,300 rows in 18 layers:
//   195-202 us, 4.6-4.7 TB/s; 64 users' long conversations in one layer: 95 us, 4.0 TB/s (a plain read of as much
//   reaches 5.8 to 6.2).  A second tile of K on its way takes registers that are not there (232-278 us for then 209).
// - More columns: 4 waves share tiles of 32 rows, which are turned into bf16 on the way into LDS, four tiles a step,
//   the next step's codes on their way meanwhile (loaded when they are needed: 273 us where this took 141,
//   drafted tokens; 102-109 now).  Bound: matrix and vector units in turn.
// - Four column blocks, over tiles that all columns see: a pipeline of its own, where each wave forms the next tile's
//   scores beside this one's weights.  4,000 tokens over 32,300 rows: 2.16 ms, 1.04 PFLOP/s, matrix cores 47% busy while
//   the clock falls to 2.07 GHz; 2.36 ms without it.  For two blocks it gains nothing.  It needs 16 rows in one page: pages
//   of 4 or 8 rows take 2.38 ms where those of 16 to 256 take 2.21.
//
// One kernel for all of them has registers for none to spare: 16 vector registers spill with bf16 output, 22 with fp32 (68 and
// 92 bytes of scratch a lane).
#include "attend_core.hpp"
#include "cache4.hpp"

namespace msa {
namespace {

// Costs: where all shares had as many tiles, those of memory rows ended after 128 us, those of local ones (four times
// the softmax, and codes to turn) after 173 to 231; one token over 4,300 + 32,000 rows in 18 layers 201 us, 217 with equal
// costs, 207 with 3 to 4, 202 with 3 to 5, 213 with 1 to 2.  Elsewhere against equal costs: 4,300 + 4,300 rows 92.5 and
// 106 us, 4,300 + 400 76 and 78.5, 16 users in four layers 173 and 179, 64 users in one 95.9 and 96.4.
struct Rows4 {
  static constexpr int kStreamCtx = 16, kStreamLocal = 64, kCtxCost = 2, kLocalCost = 3;
  static constexpr bool kLongestFirst = true;
};

// A share of the streams; `tile` is the wave's.
template <bool BF16_OUT>
__device__ __forceinline__ void attend_streams(const AttendArgs& a, Lengths& n, Plan p, Segment* seg, uint32_t* n_seg,
                                               uint16_t* tile, uint32_t number, int64_t layer, int tid) {
  constexpr int PARTS = BF16_OUT ? 1 : 3;
  constexpr int kCtx = Rows4::kStreamCtx, kLocal = Rows4::kStreamLocal;
  static_assert(kCtx == 16 && kLocal == 64, "either fits 4 loads of K and of V a lane");
  const int lane = tid & 63, wave = tid >> 6;
  const int j = lane & 15, g = lane >> 4;
  auto uni = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };
  // a local tile's V: codes as they were loaded, and 32 rows at a time turned into bf16
  constexpr int kRawBytes = kLocal * kCodes4, kTileAt = kStage * 16 - 32 * kVStride * 2;
  static_assert(kTileAt >= kRawBytes && kTileAt % 16 == 0, "both fit a stage");
  u32x4* raw = reinterpret_cast<u32x4*>(tile);
  uint16_t* vtile = tile + kTileAt / 2;

  const int32_t max_ctx = kept(a.max_ctx), shift = kept(a.page_shift);
  const char *ctx_k = kept((const char*)a.ctx_k), *ctx_v = kept((const char*)a.ctx_v);
  const int64_t ctx_row = kept(layer * a.n_groups * (int64_t)a.max_ctx);
  const int64_t layer_at = ((layer * a.n_pages) << shift) * kRow4;
  const char *page_k = kept((const char*)a.k_pages + layer_at), *page_v = kept((const char*)a.v_pages + layer_at);

  for (uint32_t from = 0;;) {
    if (tid < 3) n_seg[tid] = 0;
    __syncthreads();
    const uint32_t reached = list_segments<Rows4>(a, n, p, seg, n_seg, number, from);
    const int32_t ns = uni((int32_t)n_seg[0]);
    __syncthreads();                              // the lengths' memory becomes the tiles'

    // Two cursors run ahead of the tile that is used, across the pieces: `w` finds rows (lane r the r-th
    // of the tile), one tile later they are loaded, one tile later used.
    struct Cursor {
      int32_t s, tile, tile1, nctx, c, p0, p1, seq, grp, head;
    } w, l;
    auto enter = [&](Cursor& u, int32_t s) __attribute__((always_inline)) {
      u.s = s;
      if (s >= ns) return;
      const Segment& z = seg[s];
      u.tile = uni(z.tile0);
      u.tile1 = uni(z.tile1);
      u.c = uni(z.x.c);
      u.nctx = (u.c + kCtx - 1) / kCtx;
      u.p0 = uni(z.x.p0);
      u.p1 = uni(z.x.p1);
      u.seq = uni(z.x.seq);
      u.grp = uni(z.x.grp);
      u.head = uni(z.set * kWaves + wave);
    };
    auto step = [&](Cursor& u) __attribute__((always_inline)) {
      if (++u.tile >= u.tile1) enter(u, u.s + 1);
    };
    // The tile's row for lane r (copies of the last behind it), and its page as it stands in the table: nothing is done
    // with that before its rows are loaded, else it would be waited for, and all loads before it.
    auto row_of = [&](const Cursor& u) __attribute__((always_inline)) -> int32_t {
      if (u.tile < u.nctx) return min(u.tile * kCtx + j, u.c - 1);
      return max(0, min(u.p0 + (u.tile - u.nctx) * kLocal + lane, u.p1 - 1));
    };
    auto find = [&](const Cursor& u) __attribute__((always_inline)) -> int32_t {
      return u.tile < u.nctx ? 0 : a.page_table[(int64_t)u.seq * a.max_pages + (row_of(u) >> shift)];
    };
    // Memory tile: pk[i], pv[i] hold row 4 i + g, dims 8 j ...  Local tile: codes of row 16 i + j, dims 32 g ..,
    // and sk[i], sv[i] the scales of its four blocks (of a memory tile: nothing, but loaded all the same).
    u32x4 pk[4], pv[4];
    uint32_t sk[4], sv[4];
    auto load = [&](const Cursor& u, int32_t where) __attribute__((always_inline)) {
      const bool ctx = u.tile < u.nctx;           // uniform, as all but `rows` and `row`
      const int32_t lr = row_of(u);
      const int32_t rows = ctx ? lr : (clampi(where, 0, a.n_pages - 1) << shift) + (lr & ((1 << shift) - 1));
      const char *kb = ctx ? ctx_k : page_k, *vb = ctx ? ctx_v : page_v;
      const int64_t base = ctx ? 2 * ((ctx_row + u.grp * (int64_t)max_ctx) * kRow + u.head * kDim) : (int64_t)(u.head * kCodes4 << shift);
      const int64_t scales = ctx ? base : (int64_t)(kHeads * kCodes4 << shift) + (u.head * kBlocks4 << shift);
      const int by = ctx ? 31 : shift, step_hi = ctx ? 0 : kRow4 << shift, step_lo = ctx ? 2 * kRow : kCodes4;
      const int step_s = ctx ? 2 * kRow : kBlocks4, first = ctx ? g : j, each = ctx ? 4 : 16, at = 16 * (ctx ? j : g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t row = __shfl(rows, each * i + first, 64);
        const int64_t page = (int64_t)(row >> by) * step_hi;
        const int64_t r = (int64_t)(row & (int32_t)((1u << by) - 1u));
        pk[i] = *reinterpret_cast<const u32x4*>(kb + base + page + r * step_lo + at);
        pv[i] = *reinterpret_cast<const u32x4*>(vb + base + page + r * step_lo + at);
        sk[i] = *reinterpret_cast<const uint32_t*>(kb + scales + page + r * step_s);
        sv[i] = *reinterpret_cast<const uint32_t*>(vb + scales + page + r * step_s);
      }
    };
    // rows of the cursor's tile, or more (0: none)
    auto rows_of = [&](const Cursor& u) __attribute__((always_inline)) {
      return u.tile < u.nctx ? u.c - u.tile * kCtx : max(0, u.p1 - u.p0) - (u.tile - u.nctx) * kLocal;
    };
    u32x4 qn[4];                                  // the next piece's columns: dims 32 g + 8 d ..
    auto load_q = [&](int32_t s) __attribute__((always_inline)) {
      const Column y = column_of(a, seg[s].x, layer, seg[s].set * kWaves + wave, j);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        qn[d] = u32x4{0u, 0u, 0u, 0u};
        if (y.live) qn[d] = *reinterpret_cast<const u32x4*>(a.q + y.row * kDim + 32 * g + 8 * d);
      }
    };
    // The loaded tile; `then` once its registers have been used.
    auto attend_tile = [&](auto care, bool ctx, int32_t rows, int32_t left, const u32x4* qf, State16& st,
                           auto&& then) __attribute__((always_inline)) {
      constexpr bool CAREFUL = decltype(care)::value;
      f32x4 s[4];
      uint32_t sp = 0;                            // scales of V
      if (ctx) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<u32x4*>(tile + (4 * i + g) * kKStride + 8 * j) = pk[i];
          if (rows < kCtx && 4 * i + g >= rows) pv[i] = u32x4{0u, 0u, 0u, 0u};     // copies of the last row: weight 0
          *reinterpret_cast<u32x4*>(vtile + (4 * i + g) * kVStride + 8 * j) = pv[i];
        }
        s[0] = s[1] = s[2] = s[3] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < 4; ++d) s[0] = mfma16(*reinterpret_cast<const u32x4*>(tile + j * kKStride + 32 * g + 8 * d), qf[d], s[0]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = scale4(sk[i] >> (8 * g) & 255u);
          s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int d = 0; d < 4; ++d) s[i] = mfma16(values4(pk[i][d], f), qf[d], s[i]);
          raw[64 * i + lane] = pv[i];
          sp |= (sv[i] >> (8 * g) & 255u) << (8 * i);
        }
      }
      then();
      if (ctx) {
        attend_scored16<PARTS, CAREFUL>(vtile, s[0], left, a.scale2, lane, st);
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q > 0 && rows <= 32) continue;      // uniform
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const u32x4 codes = raw[64 * (2 * q + i) + lane];
            const float f = scale4((sp >> (16 * q + 8 * i)) & 255u);
#pragma unroll
            for (int d = 0; d < 4; ++d)
              *reinterpret_cast<u32x4*>(vtile + (16 * i + j) * kVStride + 32 * g + 8 * d) = values4(codes[d], f);
          }
          attend_scored<PARTS, CAREFUL>(vtile, s + 2 * q, left - 32 * q, a.scale2, lane, st);
        }
      }
    };
    enter(l, 0);
    w = l;
    int32_t where = 0;
    if (l.s < ns) {
      load(l, find(l));
      load_q(0);
      step(w);
      if (w.s < ns) where = find(w);
    }
    while (l.s < ns) {
      const int32_t s = l.s;
      // first local row (from p0) that the column does not see
      int32_t limit = 0;
      if (seg[s].x.p1 > seg[s].x.p0) {
        const Column y = column_of(a, seg[s].x, layer, 0, j);
        limit = seg[s].limit0 + (y.t - seg[s].x.t0);
        if (seg[s].x.shared && y.live) {
          int32_t lo = 0, hi = a.B - 1;           // the token's sequence
          while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (a.q_off[mid + 1] <= y.t) lo = mid + 1;
            else hi = mid;
          }
          limit = visible_rows(a.kv_len[lo], a.q_off[lo + 1], y.t);
        }
      }
      auto left_of = [&](const Cursor& u, int32_t rows) __attribute__((always_inline)) {
        return u.tile < u.nctx ? rows : min(rows, limit - (u.tile - u.nctx) * kLocal);
      };
      u32x4 qf[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) qf[d] = qn[d];
      State16 st;
      clear(st);
      while (l.s == s) {
        const int32_t rows = rows_of(l);
        attend_tile(std::false_type(), l.tile < l.nctx, rows, left_of(l, rows), qf, st, [&]() __attribute__((always_inline)) {
          l = w;
          if (l.s < ns) {
            load(l, where);
            if (l.s != s) load_q(l.s);
            step(w);
            if (w.s < ns) where = find(w);
          }
        });
      }
      if (needs_care(st)) {
        clear(st);
        Cursor u = l;
        enter(u, s);
#pragma unroll 1
        for (; u.tile < u.tile1; ++u.tile) {
          load(u, find(u));
          const int32_t rows = rows_of(u);
          attend_tile(std::true_type(), u.tile < u.nctx, rows, left_of(u, rows), qf, st, [] {});
        }
        if (l.s < ns) load(l, find(l));           // the next piece's first tile again
      }
      const Job job = seg[s].x;
      const Column y = column_of(a, job, layer, seg[s].set * kWaves + wave, j);
      if (seg[s].first && wave == 0 && y.live && g == 0 && (j & (a.G - 1)) == 0)
        describe(a, job, y, layer, seg[s].parts, 0, 1, kWaves, j);
      const int32_t slot = uni(seg[s].slot);
      write_state<BF16_OUT>(a, st, rows4_sum(st.l), y, layer, slot < 0 ? -1 : kWaves * slot + wave, lane);
    }
    if (reached == 0) return;                     // uniform
    from = reached;
    __syncthreads();
    load_lengths(a, n, layer, tid);
    p = plan_of<Rows4>(a, n, layer, tid);
  }
}

// ------------------------------------------------------------------ more columns

// An item: four tiles a step, brought to the four stages, then used.
template <bool BF16_OUT>
__device__ __forceinline__ void attend_item(const AttendArgs& a, const Lengths& n, ItemShared& z, u32x4* stage0, u32x4* stage1,
                                            u32x4* stage2, u32x4* stage3, int64_t layer, int tid) {
  constexpr int PARTS = BF16_OUT ? 1 : 3;
  auto uni = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };
  const int lane = tid & 63, wave = uni(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const Item& it = z.item;
  const Job x = it.x;
  // fewer column blocks than waves: `share` waves take a block's columns and the tiles in turn
  const int32_t blocks = uni(it.blocks), unit = uni(it.unit), share = kWaves / blocks;
  const int32_t tile0 = uni(it.tile0), head = uni(it.head);
  int32_t tile1 = uni(it.tile1);
  const int cb = wave & (blocks - 1), turn = uni(wave / blocks);
  const Column y = column_of(a, x, layer, head, it.col0 + cb * kCols + c);
  int32_t limit = 0;                                 // first local row (from p0) the column does not see
  if (y.live && x.p1 > x.p0) {
    const int32_t b = x.shared ? min(count_upto(n.off, a.B, y.t), a.B - 1) : x.seq;
    limit = clampi(visible_rows(n.len[b], n.off[b + 1], y.t) - x.p0, 0, x.p1 - x.p0);
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
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    qf[d] = u32x4{0u, 0u, 0u, 0u};
    if (y.live) qf[d] = *reinterpret_cast<const u32x4*>(a.q + y.row * kDim + 16 * d + 8 * h);
  }
  if (it.first && turn == 0 && y.live && h == 0 && (c & (a.G - 1)) == 0)
    describe(a, x, y, layer, it.parts, it.unit < 0 ? 0 : kBlockUnits * cb, it.width, it.width * kHeads, c);
  if (lane == 0) {
    z.most[wave] = most;
    z.least[wave] = least;
  }
  __syncthreads();                                   // the lengths' memory becomes the tiles'

  const int32_t jc = uni(x.c), p0 = uni(x.p0), seq = uni(x.seq), nctx = (jc + kTileRows - 1) / kTileRows;
  int32_t wg_most = 0, wg_least = 0x7FFFFFFF;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    wg_most = max(wg_most, z.most[w]);
    wg_least = min(wg_least, z.least[w]);
  }
  wg_most = uni(wg_most);
  wg_least = uni(wg_least);
  tile1 = min(tile1, nctx + (wg_most + kTileRows - 1) / kTileRows);

  const int64_t ctx_at = (layer * a.n_groups + uni(x.grp)) * (int64_t)a.max_ctx * kRow + head * kDim;
  const int64_t layer_at = ((layer * a.n_pages) << a.page_shift) * kRow4;
  const uint16_t *ctx_k = a.ctx_k + ctx_at, *ctx_v = a.ctx_v + ctx_at;
  const int32_t shift = kept(a.page_shift);
  // a local tile's blocks, one a thread: waves 0 and 1 K, 2 and 3 V; row br of the tile, dims 32 bb ..
  const uint8_t* pages = (const uint8_t*)(wave < 2 ? a.k_pages : a.v_pages) + layer_at;
  const int br = 16 * (wave & 1) + (lane >> 2), bb = lane & 3;
  // where its chunk d lies in a stage: chunk 4 bb + d permuted as the reads expect
  const int lds_row = (wave < 2 ? 0 : kTileRows * 16) + br * 16 + 4 * (bb ^ (wave < 2 ? (br >> 2) & 3 : br & 3));
  // The four local tiles from t on (the last row again behind it): their pages, a step later their codes and scales.
  auto local_of = [&](int32_t t, int i) __attribute__((always_inline)) {
    return p0 + min((t + i - nctx) * kTileRows + br, wg_most - 1);
  };
  auto find_local = [&](int32_t t, int32_t* page) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) page[i] = a.page_table[(int64_t)seq * a.max_pages + (local_of(t, i) >> shift)];
  };
  auto load_local = [&](int32_t t, const int32_t* page, u32x4* raw, uint32_t* scales) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t r = local_of(t, i) & ((1 << shift) - 1);
      const uint8_t* p = pages + (int64_t)clampi(page[i], 0, a.n_pages - 1) * (kRow4 << shift);
      raw[i] = *reinterpret_cast<const u32x4*>(p + codes4_at(head, r, shift) + 16 * bb);
      scales[i] = *reinterpret_cast<const uint32_t*>(p + scales4_at(head, r, shift));      // of the row's four blocks
    }
  };
  auto put_local = [&](u32x4 raw, uint32_t scales, u32x4* stage) __attribute__((always_inline)) {
    const float f = scale4(scales >> (8 * bb) & 255u);
#pragma unroll
    for (int d = 0; d < 4; ++d) stage[lds_row + (d ^ (br & 3))] = values4(raw[d], f);
  };
  auto fill_ctx = [&](int32_t t, u32x4* stage) __attribute__((always_inline)) {
    t = min(t, nctx - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * wave + 4 * i + (lane >> 4);
      const int64_t at = (int64_t)min(t * kTileRows + r, jc - 1) * kRow;
      u32x4* to = stage + 16 * (8 * wave + 4 * i);
      __builtin_amdgcn_global_load_lds((gptr_t)(ctx_k + at + 8 * ((lane & 15) ^ (r & 15))), (lptr_t)to, 16, 0, 0);
      __builtin_amdgcn_global_load_lds((gptr_t)(ctx_v + at + 8 * ((lane & 15) ^ (5 * (r & 3)))),
                                       (lptr_t)(to + kTileRows * 16), 16, 0, 0);
    }
  };
  StageReads at(lane);
  State st;
  clear(st);
  // rows of tile t that a column sees, or more; whether all the wave's columns see all of it
  auto left_of = [&](int32_t t) __attribute__((always_inline)) {
    return t >= tile1 ? 0 : (t < nctx ? jc - t * kTileRows : limit - (t - nctx) * kTileRows);
  };
  const int32_t odd = jc & (kTileRows - 1) ? nctx - 1 : -1, whole_end = nctx + min(wg_most, least) / kTileRows;
  auto whole = [&](int32_t t) __attribute__((always_inline)) { return t != odd && t < whole_end; };
  const uint32_t a0 = lds_at(stage0), a1 = lds_at(stage1), a2 = lds_at(stage2), a3 = lds_at(stage3);
  // Four column blocks: whole local tiles, two a step, whose 16 rows a wave lie in one page.  A wave forms the scores of
  // its next tile while this one's turn into weights: matrix and vector work of one wave that do not wait for each
  // other.  So K is a tile ahead of V, and LDS holds K and V of four tiles, two that are read and two that are
  // written.  Codes are on their way for a step before they are turned into bf16.
  auto units = [&](int32_t first, int32_t n) __attribute__((always_inline)) {
    // Pages by vector loads, of one address: a scalar load on its way would make every wait for LDS a wait for all of it.
    // Row addresses are in scalar registers.
    const int32_t* table = kept(a.page_table + (int64_t)seq * a.max_pages);
    const int zero = threadIdx.x >> 8;            // 0, but not to the compiler
    typedef const __attribute__((address_space(1))) uint8_t* pool_t;
    const pool_t all_k = (pool_t)kept((const uint8_t*)a.k_pages + layer_at), all_v = (pool_t)kept((const uint8_t*)a.v_pages + layer_at);
    const int32_t last_page = kept(a.n_pages - 1), page_bytes = kept(kRow4 << shift);
    const int32_t head_codes = kept(codes4_at(head, 0, shift)), head_scales = kept(scales4_at(head, 0, shift));
    const int32_t row_w = uni(p0 + (first - nctx) * kTileRows + 16 * wave);
    const int32_t last_row = uni(p0 + (first - nctx + 2 * n - 1) * kTileRows + 16 * (wave & 1));
    // first of this wave's 16 rows of tiles t and t + 1 (t from `first` on; the last tile again behind it)
    auto row_of = [&](int32_t t) __attribute__((always_inline)) { return min(row_w + t * kTileRows, last_row); };
    auto find = [&](int32_t t) __attribute__((always_inline)) -> int32_t { return table[(row_of(t) >> shift) + zero]; };
    struct Raw {
      u32x4 codes;
      uint32_t scales;       // of the row's four blocks (a byte's extension would be waited for long before its use)
    };
    auto load = [&](pool_t pool, int32_t t, int32_t page) __attribute__((always_inline)) -> Raw {
      const int32_t r = row_of(t) & ((1 << shift) - 1);
      const pool_t p = pool + (int64_t)clampi(uni(page), 0, last_page) * page_bytes;
      const pool_t codes = p + (head_codes + r * kCodes4), scales = p + (head_scales + r * kBlocks4);
      Raw x;
      x.codes = *(const __attribute__((address_space(1))) u32x4*)(codes + (uint32_t)(16 * lane));
      x.scales = *(const __attribute__((address_space(1))) uint32_t*)(scales + (uint32_t)(4 * (lane >> 2)));
      return x;
    };
    // a tile's place: K in stages 0 and 1, V in 2 and 3, of four tiles in turn
    auto slot = [&](int32_t t) __attribute__((always_inline)) { return (uint32_t)(8192 * (t & 3)); };
    const int part = br * 16, at_k = part + 4 * (bb ^ ((br >> 2) & 3)), at_v = part + 4 * (bb ^ (br & 3));
    const uint32_t to_k = 16 * (at_k + (br & 3)), to_v = 16 * (at_v + (br & 3));
    auto put = [&](uint32_t base, uint32_t to, const Raw& x) __attribute__((always_inline)) {
      const float f = scale4(x.scales >> (8 * bb) & 255u);
#pragma unroll
      for (int d = 0; d < 4; ++d) *const_cast<u32x4*>(lds_ptr((to ^ (16 * d)) + base)) = values4(x.codes[d], f);
    };
    // waves 0 and 1 bring the first tile of two, 2 and 3 the second
    const int32_t second = wave >> 1;
    // K of tiles 0 to 2, V of 0 and 1
    {
      const Raw k0 = load(all_k, 0, find(0)), k1 = load(all_k, 1, find(1)), v0 = load(all_v, 0, find(0));
      if (second == 0) put(a0 + slot(0), to_k, k0);
      put(a0 + (second ? slot(2) : slot(1)), to_k, k1);
      put(a2 + (second ? slot(1) : slot(0)), to_v, v0);
    }
    // step u brings K of tiles 2 u + 3 and the next, V of 2 u + 2 and the next
    Raw rk = load(all_k, 3, find(3)), rv = load(all_v, 2, find(2));
    int32_t page_k = find(5), page_v = find(4);
    auto form = [&](uint32_t at_slot) __attribute__((always_inline)) {
      f32x16 s = zeros16();
#pragma unroll
      for (int d = 0; d < 8; ++d) s = mfma32(at.k(lds_ptr(a0 + at_slot), d), qf[d], s);
      return s;
    };
    __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt 0
    asm volatile("s_barrier" ::: "memory");
    f32x16 s = form(0);
    float top = halves_max(max16(s));
    // the tile whose scores are formed: its V at v_slot; the next one's K at k_slot
    auto tile = [&](uint32_t k_slot, uint32_t v_slot) __attribute__((always_inline)) {
      u32x4 kf[8], vf[2][4];
#pragma unroll
      for (int d = 0; d < 8; ++d) kf[d] = at.k(lds_ptr(a0 + k_slot), d);
      __builtin_amdgcn_sched_barrier(0);
      raise_to<false>(top, a.scale2, st);
      auto read_v = [&](int m) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < 4; ++d)      // V rows lie behind a stage's 32 K rows for `v`, 8 KB
          vf[m][d] = at.v(lds_ptr(a2 + v_slot - 8192), m, d);
        __builtin_amdgcn_sched_barrier(0);
      };
      u32x4 pw[2][PARTS];
      auto weigh = [&](int m) __attribute__((always_inline)) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s[8 * m + e];
        weights<PARTS, false>(v, a.scale2, st.neg, pw[m], st.l);
      };
      auto sum = [&](int m) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < 4; ++d) add_values<PARTS, false>(vf[m][d], pw[m], st.o[d]);
      };
      read_v(0);
      f32x16 t = zeros16();
#pragma unroll
      for (int d = 0; d < 8; ++d) t = mfma32(kf[d], qf[d], t);
      weigh(0);
      weigh(1);
      s = t;
      read_v(1);
      sum(0);
      sum(1);
      top = halves_max(max16(s));
    };
    // u even: i = 0
    auto step = [&](auto odd_u, int32_t u) __attribute__((always_inline)) {
      constexpr int i = decltype(odd_u)::value, T = 2 * i;       // its first tile, of four
      __builtin_amdgcn_s_waitcnt(0xC07F);         // this wave's part of the next tiles is written
      asm volatile("s_barrier" ::: "memory");
      tile(8192 * (T + 1), 8192 * T);
      put(a0 + 8192 * (second ? T : (T + 3) & 3), to_k, rk);
      put(a2 + 8192 * (second ? (T + 3) & 3 : (T + 2) & 3), to_v, rv);
      rk = load(all_k, 2 * u + 5, page_k);
      rv = load(all_v, 2 * u + 4, page_v);
      page_k = find(2 * u + 7);
      page_v = find(2 * u + 6);
      tile(8192 * ((T + 2) & 3), 8192 * (T + 1));
    };
#pragma unroll 1
    for (int32_t u = 0; u + 1 < n; u += 2) {      // pairs: each step's loads are always followed by the other's
      step(std::integral_constant<int, 0>(), u);
      step(std::integral_constant<int, 1>(), u + 1);
    }
    if (n & 1) step(std::integral_constant<int, 0>(), n - 1);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");
  };
  auto pass = [&](auto care) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(care)::value;
    auto use = [&](int32_t t, int32_t end) __attribute__((always_inline)) {
#pragma unroll 1
      for (int i = turn; i < 4; i += share) {
        if (t + i >= end) break;
        const u32x4* s = lds_ptr(i == 0 ? a0 : (i == 1 ? a1 : (i == 2 ? a2 : a3)));
        attend_tiles<PARTS, CAREFUL, 1>(nullptr, s, s, at, qf, t + i, whole(t + i), left_of, a.scale2, h, st);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);         // what was read of the tiles is in registers
      asm volatile("s_barrier" ::: "memory");
    };
    const int32_t ctx_end = min(tile1, nctx);
    int32_t local0 = max(tile0, nctx);
#pragma unroll 1
    for (int32_t t = tile0; t < ctx_end; t += 4) {
      fill_ctx(t, stage0);
      fill_ctx(t + 1, stage1);
      fill_ctx(t + 2, stage2);
      fill_ctx(t + 3, stage3);
      __builtin_amdgcn_s_waitcnt(0x70);           // vmcnt, lgkmcnt 0
      __syncthreads();
      use(t, ctx_end);
    }
    if (!CAREFUL && blocks == kWaves && shift >= 4 && (p0 & 15) == 0) {
      const int32_t tiles = min(tile1, nctx + min(wg_most, wg_least) / kTileRows) - local0, n = tiles / 2;
      if (n > 0) {
        units(local0, n);
        local0 += 2 * n;
      }
    }
    int32_t page[4];
    u32x4 raw[4];
    uint32_t scales[4];
    if (local0 < tile1) {
      find_local(local0, page);
      load_local(local0, page, raw, scales);
      find_local(local0 + 4, page);
    }
#pragma unroll 1
    for (int32_t t = local0; t < tile1; t += 4) {
      put_local(raw[0], scales[0], stage0);
      put_local(raw[1], scales[1], stage1);
      put_local(raw[2], scales[2], stage2);
      put_local(raw[3], scales[3], stage3);
      if (t + 4 < tile1) {
        load_local(t + 4, page, raw, scales);
        find_local(t + 8, page);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);         // lgkmcnt 0: the tiles are written; the next ones stay on their way
      asm volatile("s_barrier" ::: "memory");
      use(t, tile1);
    }
  };
  pass(std::false_type());
  if (__syncthreads_or(needs_care(st))) {
    clear(st);
    pass(std::true_type());
  }
  finish_item<BF16_OUT>(a, z, st, y, layer, unit, blocks, cb, turn, wave, lane, stage1, stage2, stage3);
}

template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads, 2)
attend4_kernel(const AttendArgs a) {
  __shared__ u32x4 stages[4 * kStage];
  u32x4 *const stage0 = stages, *const stage1 = stages + kStage, *const stage2 = stages + 2 * kStage, *const stage3 = stages + 3 * kStage;
  __shared__ union {
    ItemShared item;
    struct {
      Segment seg[kSegments];
      uint32_t n_seg[3];
    } streams;
  } sh;
  const int tid = threadIdx.x;
  // layers fastest: the workgroups that turn out to have nothing to do come last
  const int64_t layer = blockIdx.x;
  const uint32_t id = blockIdx.z * gridDim.y + blockIdx.y;
  if (a.plans && id >= a.plans[layer * kThreads].shares + a.plans[layer * kThreads].all_items) return;
  Lengths n = lengths_in(stage0, stage1, stage2, stage3);
  load_lengths(a, n, layer, tid);
  const Plan p = plan_of<Rows4>(a, n, layer, tid);
  // items that fit the chip at once are the longer ones; items of many rounds end more evenly than shares
  const bool items_first = p.all_items <= (uint32_t)a.both_wgs;
  const uint32_t first_share = items_first ? p.all_items : 0, first_item = items_first ? 0 : p.shares;
  if (id >= first_share && id < first_share + p.shares) {      // uniform
    const int wave = tid >> 6;
    u32x4* tile = wave == 0 ? stage0 : (wave == 1 ? stage1 : (wave == 2 ? stage2 : stage3));
    attend_streams<BF16_OUT>(a, n, p, sh.streams.seg, sh.streams.n_seg, reinterpret_cast<uint16_t*>(tile),
                             id - first_share, layer, tid);
  } else if (id >= first_item && id < first_item + p.all_items) {
    // Items of one round, two a CU: the longest that need not share have a CU each, of the others the longest and the shortest
    // are side by side.  CUs then end within 85 to 98 us, 59 to 124 without.  A pair is layers * (512 / layers / 2) workgroups
    // apart, the number of CUs where the layers divide that, else a few less: sequences of drafted tokens in 1, 2 and 4 layers
    // 103, 118 and 109 us (107, 123 and 113 unpaired), three in 18 layers 332 (334), 24 in one layer 57.6 (56.9).
    uint32_t item = id - first_item;
    const uint32_t cus = a.wgs / 2, n_items = p.all_items;
    if (p.all_cost == 0 && n_items > cus && n_items <= 2 * cus) {
      const uint32_t alone = 2 * cus - n_items;
      item = item < cus - alone ? item + alone : (item < cus ? item - (cus - alone) : n_items - 1 - (item - cus));
    }
    find_item(a, n, p, sh.item.item, item, tid);
    if (sh.item.item.valid) attend_item<BF16_OUT>(a, n, sh.item, stage0, stage1, stage2, stage3, layer, tid);
  }
}

}  // namespace

hipError_t launch_attend4(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* q,
                          const int32_t* q_off, const int32_t* grp_off, const uint16_t* ctx_k, const uint16_t* ctx_v,
                          const int32_t* ctx_len, int32_t max_ctx, const uint8_t* k_pages, const uint8_t* v_pages,
                          int32_t n_pages, int32_t page_shift, const int32_t* page_table, int32_t max_pages,
                          const int32_t* kv_len, const int32_t* pre_len, float scale, bool bf16_out, void* out,
                          void* ws, hipStream_t s) {
  if (!can_share(B)) grp_off = nullptr;      // one sequence, so one group
  const Sizes z = sizes_of(L, B, n_groups, n_q, Hq / kHeads, grp_off != nullptr);
  const AttendArgs a = args_of(z, B, n_groups, n_q, Hq, q, q_off, grp_off, ctx_k, ctx_v, ctx_len, max_ctx, k_pages, v_pages,
                               n_pages, page_shift, page_table, max_pages, kv_len, pre_len, scale, out, ws);
  if (bf16_out) launch_as<Rows4, true>(attend4_kernel<true>, a, z, L, s);
  else launch_as<Rows4, false>(attend4_kernel<false>, a, z, L, s);
  return hipGetLastError();
}

}  // namespace msa
