// attend.hip -- attention of ragged new tokens over [memory context ; paged local rows], the
// context and the first local pages shared by the sequences of a group.
//
// For every layer, token i of sequence b (n_b new tokens) in group g sees the group's memory rows
// 0 .. ctx_len[g]) and its local rows 0 .. kv_len[b] - n_b + i; query head hq reads KV head
// hq / (Hq / 8); the output is the softmax-weighted sum of the visible V rows.
//
// The work is a list of jobs, each of columns over rows (attend_core.hpp).
//
// One kernel (attend_kernel) whose workgroups are of two kinds, so that both fill the chip together:
// - jobs of up to 16 columns are bound by the rows' bytes: a wave takes one KV head and streams rows
//   through a tile of its own in LDS, without barriers (attend_streams);
// - more columns are bound by the matrix cores and the softmax's vector work: 4 waves take one head and
//   share each tile of 32 rows, 32 columns a wave (attend_item).
// attend_join_kernel joins where a column's rows were cut into parts; what is whole in one part has been
// written by the workgroup that computed it.  (A workgroup that joins for the others would need a counter and
// a device-wide release in each; the launch costs ~5 us.)
// Measured: one token of 32 heads over 4,364 rows in 18 layers 61-73 us (4.1-4.9 TB/s); a prompt of 8,000 tokens over
// 4,300 memory rows 1.03-1.12 ms (960-1,044 TFLOP/s, bf16 output).  There the matrix cores are 50% busy and the
// vector units 44%; they overlap little, every instruction between a tile's barrier and its last product
// shows in the time, and the clock gives way as the work gets denser (2.16 GHz at 1.18 ms, 1.94 at 1.07).
// In both, S^T = K . Q^T is computed with K as the A operand and the columns as the B operand
// (registers), so a lane holds scores of one column and the softmax needs only exchanges between the
// lane groups of a wave; for O^T += V^T . P^T the MFMA's k axis is taken in the order in which the scores
// already lie in the lanes, and V^T comes from the row-major tile by transposed LDS reads.  Scores,
// running maximum (log2 units), sum and output are fp32.
#include "attend_core.hpp"

namespace msa {
namespace {

// A share of the streams; `tile` is the wave's.
template <bool BF16_OUT>
__device__ __forceinline__ void attend_streams(const AttendArgs& a, Lengths& n, Plan p, Segment* seg, uint32_t* n_seg,
                                               uint16_t* tile, uint32_t number, int64_t layer, int tid) {
  constexpr int PARTS = BF16_OUT ? 1 : 3;
  static_assert(kStage * 16 >= kStreamRows * kVStride * 2, "a stage holds a wave's tile");
  const int lane = tid & 63, wave = tid >> 6;
  // rows by whole 16-lane groups: load i brings rows 4 i + g, dims 8 j .. 8 j + 7
  const int j = lane & 15, g = lane >> 4;
  auto uni = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };

  const uint16_t *ctx_k = kept(a.ctx_k), *ctx_v = kept(a.ctx_v), *page_k = kept((const uint16_t*)a.k_pages),
                 *page_v = kept((const uint16_t*)a.v_pages);
  const int32_t max_ctx = kept(a.max_ctx);
  const int64_t ctx_row = kept(layer * a.n_groups * (int64_t)a.max_ctx);
  const int64_t page_row0 = kept((layer * a.n_pages) << a.page_shift);

  for (uint32_t from = 0;;) {
    if (tid < 3) n_seg[tid] = 0;
    __syncthreads();
    const uint32_t reached = list_segments<RowsBf16>(a, n, p, seg, n_seg, number, from);
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
      u.nctx = (u.c + kStreamRows - 1) / kStreamRows;
      u.p0 = uni(z.x.p0);
      u.p1 = uni(z.x.p1);
      u.seq = uni(z.x.seq);
      u.grp = uni(z.x.grp);
      u.head = uni(z.set * kWaves + wave);
    };
    auto step = [&](Cursor& u) __attribute__((always_inline)) {
      if (++u.tile >= u.tile1) enter(u, u.s + 1);
    };
    auto find = [&](const Cursor& u) __attribute__((always_inline)) -> int32_t {
      const int32_t r = lane & 31;
      if (u.tile < u.nctx) return min(u.tile * kStreamRows + r, u.c - 1);
      return u.p1 > u.p0 ? page_row(a, u.seq, min(u.p0 + (u.tile - u.nctx) * kStreamRows + r, u.p1 - 1)) : 0;
    };
    u32x4 pk[8], pv[8];
    auto load = [&](const Cursor& u, int32_t where) __attribute__((always_inline)) {
      const bool ctx = u.tile < u.nctx;
      const int64_t base = (ctx ? (ctx_row + u.grp * (int64_t)max_ctx) : page_row0) * kRow + u.head * kDim;
      const uint16_t* kb = (ctx ? ctx_k : page_k) + base;
      const uint16_t* vb = (ctx ? ctx_v : page_v) + base;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t off = (int64_t)__shfl(where, 4 * i + g, 64) * kRow + 8 * j;
        pk[i] = *reinterpret_cast<const u32x4*>(kb + off);
        pv[i] = *reinterpret_cast<const u32x4*>(vb + off);
      }
    };
    // rows of the cursor's tile, or more (0: none)
    auto rows_of = [&](const Cursor& u) __attribute__((always_inline)) {
      return u.tile < u.nctx ? u.c - u.tile * kStreamRows : max(0, u.p1 - u.p0) - (u.tile - u.nctx) * kStreamRows;
    };
    auto stage_k = [&](int32_t rows) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        *reinterpret_cast<u32x4*>(tile + (4 * i + g) * kKStride + 8 * j) = pk[i];
        if (rows < kStreamRows && 4 * i + g >= rows) pv[i] = u32x4{0u, 0u, 0u, 0u};   // copies of the last row: weight 0
      }
    };
    u32x4 qn[4];                                  // the next piece's columns
    auto load_q = [&](int32_t s) __attribute__((always_inline)) {
      const Column y = column_of(a, seg[s].x, layer, seg[s].set * kWaves + wave, j);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        qn[d] = u32x4{0u, 0u, 0u, 0u};
        if (y.live) qn[d] = *reinterpret_cast<const u32x4*>(a.q + y.row * kDim + 32 * d + 8 * g);
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
      u32x4 qf[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) qf[d] = qn[d];
      State16 st;
      clear(st);
      while (l.s == s) {
        const int32_t rows = rows_of(l);
        const int32_t left = l.tile < l.nctx ? rows : min(rows, limit - (l.tile - l.nctx) * kStreamRows);
        stage_k(rows);
        attend_rows<PARTS, false>(tile, pv, qf, left, a.scale2, lane, st, [&]() __attribute__((always_inline)) {
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
        for (; u.tile < u.tile1; ++u.tile) {
          load(u, find(u));
          const int32_t rows = rows_of(u);
          stage_k(rows);
          const int32_t left = u.tile < u.nctx ? rows : min(rows, limit - (u.tile - u.nctx) * kStreamRows);
          attend_rows<PARTS, true>(tile, pv, qf, left, a.scale2, lane, st, [] {});
        }
        if (l.s < ns) load(l, find(l));           // the next piece's first tile again
      }
      const Job x = seg[s].x;
      const Column y = column_of(a, x, layer, seg[s].set * kWaves + wave, j);
      if (seg[s].first && wave == 0 && y.live && g == 0 && (j & (a.G - 1)) == 0)
        describe(a, x, y, layer, seg[s].parts, 0, 1, kWaves, j);
      const int32_t slot = uni(seg[s].slot);
      write_state<BF16_OUT>(a, st, rows4_sum(st.l), y, layer, slot < 0 ? -1 : kWaves * slot + wave, lane);
    }
    if (reached == 0) return;                     // uniform
    from = reached;
    __syncthreads();
    load_lengths(a, n, layer, tid);
    p = plan_of<RowsBf16>(a, n, layer, tid);
  }
}

// ------------------------------------------------------------------ more columns

// An item.  An array for each stage, so that the compiler sees which one an access touches.
template <bool BF16_OUT>
__device__ __forceinline__ void attend_item(const AttendArgs& a, const Lengths& n, ItemShared& z, u32x4* stage0, u32x4* stage1,
                                            u32x4* stage2, u32x4* stage3, int64_t layer, int tid) {
  constexpr int PARTS = BF16_OUT ? 1 : 3;
  const int lane = tid & 63, wave = tid >> 6;
  const int c = lane & 31, h = lane >> 5;
  const Item& it = z.item;
  auto uni = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };
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
  if (lane == 0) z.most[wave] = most;
  __syncthreads();                                   // the lengths' memory becomes the tiles'

  const int32_t jc = uni(x.c), p0 = uni(x.p0), seq = uni(x.seq), nctx = (jc + kTileRows - 1) / kTileRows;
  int32_t wg_most = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) wg_most = max(wg_most, z.most[w]);
  wg_most = uni(wg_most);
  tile1 = min(tile1, nctx + (wg_most + kTileRows - 1) / kTileRows);

  // This wave's loads: rows 8 wave + 4 i + (lane >> 4) of K and of V.  8 memory rows follow each other, and so do 8
  // local rows of a page, so one row number and fixed lane offsets address a wave's loads of a whole tile.
  // Partial tiles, and local rows that do not lie in eights (small pages, an odd start), are found row by row.
  constexpr int kPer = kTileRows / 4 / kWaves;
  const int64_t ctx_at = (layer * a.n_groups + uni(x.grp)) * (int64_t)a.max_ctx * kRow + head * kDim;
  const int64_t page_at = ((layer * a.n_pages) << a.page_shift) * kRow + head * kDim;
  const char *ctx_k = kept((const char*)(a.ctx_k + ctx_at)), *ctx_v = kept((const char*)(a.ctx_v + ctx_at));
  const char *page_k = kept((const char*)a.k_pages + 2 * page_at), *page_v = kept((const char*)a.v_pages + 2 * page_at);
  const auto* table = (const __attribute__((address_space(4))) int32_t*)kept(a.page_table + (int64_t)seq * a.max_pages);
  const int32_t shift = kept(a.page_shift), last_page = kept(a.n_pages - 1);
  const int w8 = uni(4 * kPer * wave);
  // the memory rows' partial tile, if they have one; the end of the tiles whose rows are found by eights, of
  // those that all the wave's columns see
  const int32_t odd = jc & (kTileRows - 1) ? nctx - 1 : -1;
  const int32_t eights_end = nctx + (shift >= 3 && (p0 & 7) == 0 ? wg_most / kTileRows : 0);
  const int32_t whole_end = nctx + min(wg_most, least) / kTileRows;
  uint32_t k_lane[kPer], v_lane[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = 4 * i + (lane >> 4);
    k_lane[i] = 2 * (r * kRow + 8 * ((lane & 15) ^ ((w8 + r) & 15)));
    v_lane[i] = 2 * (r * kRow + 8 * ((lane & 15) ^ (5 * (lane >> 4))));
  }
  // the page of the wave's rows of a page tile, as it stands in the table: a scalar load (a vector load's result
  // would only come after all the tile loads issued before it), not waited for before the tile's turn
  int32_t page_a = 0, page_b = 0;
  constexpr int kWaitOld = (4 * kPer) | 0x70, kWaitAll = 0x70;       // vmcnt, lgkmcnt 0
  auto local_row = [&](int32_t t) __attribute__((always_inline)) {
    return p0 + min((t - nctx) * kTileRows + w8, wg_most - 1);
  };
  auto find = [&](int32_t t, int32_t& page) __attribute__((always_inline)) {
    if (t >= nctx) page = table[local_row(t) >> shift];
  };
  auto issue = [&](int32_t t, int32_t page, u32x4* stage) __attribute__((always_inline)) {
    const bool ctx = t < nctx;
    const char *kb = ctx ? ctx_k : page_k, *vb = ctx ? ctx_v : page_v;
    u32x4* to = stage + kPer * 64 * (w8 / (4 * kPer));
    if (t != odd && t < eights_end) {
      int32_t row = t * kTileRows + w8;
      if (!ctx) row = (clampi(page, 0, last_page) << shift) + (local_row(t) & ((1 << shift) - 1));
      kb += (int64_t)row * (2 * kRow);
      vb += (int64_t)row * (2 * kRow);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        __builtin_amdgcn_global_load_lds((gptr_t)(kb + k_lane[i]), (lptr_t)(to + 64 * i), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((gptr_t)(vb + v_lane[i]), (lptr_t)(to + 64 * i + kTileRows * 16), 16, 0, 0);
      }
      asm volatile("" ::: );      // keeps the two branches' loads apart: these have scalar bases
    } else {
      int by = lane >> 4;
      asm volatile("" : "+v"(by));          // what follows is not kept in registers from tile to tile
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = 4 * i + by;
        const int32_t row = ctx ? min(t * kTileRows + w8 + r, jc - 1)
                                : page_row(a, seq, p0 + min((t - nctx) * kTileRows + w8 + r, wg_most - 1));
        const int64_t at = (int64_t)(row - r) * (2 * kRow);
        __builtin_amdgcn_global_load_lds((gptr_t)(kb + at + k_lane[i]), (lptr_t)(to + 64 * i), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((gptr_t)(vb + at + v_lane[i]), (lptr_t)(to + 64 * i + kTileRows * 16), 16, 0, 0);
      }
    }
  };
  const StageReads at(lane);
  State st;
  clear(st);
  // rows of tile t that a column sees, or more; whether all the wave's columns see all of it
  auto left_of = [&](int32_t t) __attribute__((always_inline)) {
    return t >= tile1 ? 0 : (t < nctx ? jc - t * kTileRows : limit - (t - nctx) * kTileRows);
  };
  auto whole = [&](int32_t t) __attribute__((always_inline)) {
    return t != odd && t < whole_end;
  };
  const int32_t last = tile1 - 1;
  // Four column blocks, bound by the matrix cores and the vector work: one tile a step.  This wave's loads of it
  // have landed (they were issued three tiles ago; those of the two tiles after it may be in flight: 2 x 2 kPer),
  // barrier (the tile is whole, and every wave is done with the tile before), ask for its K fragments, load
  // the tile three ahead into the stage of the one before (the fragments come meanwhile: 1.15 against
  // 1.18 ms for a prompt of 8,000 tokens), use this one.
  auto step = [&](int32_t t, const u32x4* stage, u32x4* before) __attribute__((always_inline)) {
    if (t + 2 < tile1) __builtin_amdgcn_s_waitcnt(kWaitOld);
    else __builtin_amdgcn_s_waitcnt(kWaitAll);
    asm volatile("s_barrier" ::: "memory");
    u32x4 kf[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) kf[d] = at.k(stage, d);
    if (t + 3 < tile1) {
      issue(t + 3, page_a, before);
      find(min(t + 4, last), page_a);
    }
    attend_tiles<PARTS, false, 1>(kf, stage, stage, at, qf, t, whole(t), left_of, a.scale2, h, st);
  };
  // Fewer blocks, bound by the rows' bytes: four tiles a step, one or two for each wave, and the next four only
  // once all are done: the other workgroup of the CU computes or loads meanwhile.  (Two tiles in use and two on
  // their way, one wave computing at a time: 78 us for 46 tiles of 64 columns, so 56.)  A tile behind the last
  // is a copy of it that nothing sees.
  int32_t pages[kWaves];
  auto issue_all = [&](int32_t t) __attribute__((always_inline)) {
    issue(t, pages[0], stage0);
    issue(min(t + 1, last), pages[1], stage1);
    issue(min(t + 2, last), pages[2], stage2);
    issue(min(t + 3, last), pages[3], stage3);
  };
  auto find_all = [&](int32_t t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kWaves; ++i) find(min(t + i, last), pages[i]);
  };
  auto steps = [&](auto per) __attribute__((always_inline)) {
    constexpr int N = decltype(per)::value;
    const uint32_t from = turn * N, a0 = lds_at(stage0), a1 = lds_at(stage1), a2 = lds_at(stage2), a3 = lds_at(stage3);
    const u32x4* sa = lds_ptr(from == 0 ? a0 : (from == 1 ? a1 : (from == 2 ? a2 : a3)));
    const u32x4* sb = N == 2 ? lds_ptr(from == 0 ? a1 : a3) : sa;
    for (int32_t t = tile0;; t += kWaves) {
      __builtin_amdgcn_s_waitcnt(kWaitAll);
      asm volatile("s_barrier" ::: "memory");
      const int32_t u = t + N * turn;
      if (u < tile1)
        attend_tiles<PARTS, false, N>(nullptr, sa, sb, at, qf, u, u + N - 1 < tile1 && whole(u) && whole(u + N - 1),
                                      left_of, a.scale2, h, st);
      if (t + kWaves >= tile1) break;
      asm volatile("s_barrier" ::: "memory");
      issue_all(t + kWaves);
      find_all(t + 2 * kWaves);
    }
  };
  if (tile0 < tile1) {
    if (blocks == kWaves) {
      find(tile0, page_a);
      find(min(tile0 + 1, last), page_b);
      issue(tile0, page_a, stage0);
      issue(min(tile0 + 1, last), page_b, stage1);
      find(min(tile0 + 2, last), page_a);
      find(min(tile0 + 3, last), page_b);
      if (tile0 + 2 < tile1) issue(tile0 + 2, page_a, stage2);
      page_a = page_b;
      for (int32_t t = tile0; t < tile1; t += 4) {
        step(t, stage0, stage3);
        if (t + 1 < tile1) step(t + 1, stage1, stage0);
        if (t + 2 < tile1) step(t + 2, stage2, stage1);
        if (t + 3 < tile1) step(t + 3, stage3, stage2);
      }
    } else {
      find_all(tile0);
      issue_all(tile0);
      find_all(tile0 + kWaves);
      if (blocks == 2) steps(std::integral_constant<int, 2>());
      else steps(std::integral_constant<int, 1>());
    }
  }
  if (__syncthreads_or(needs_care(st))) {
    clear(st);
#pragma unroll 1
    for (int32_t t = tile0; t < tile1; ++t) {
      find(t, page_a);
      issue(t, page_a, stage0);
      __builtin_amdgcn_s_waitcnt(kWaitAll);
      __syncthreads();
      if ((t & (share - 1)) == turn)
        attend_tiles<PARTS, true, 1>(nullptr, stage0, stage0, at, qf, t, false, left_of, a.scale2, h, st);
      __syncthreads();
    }
  }
  finish_item<BF16_OUT>(a, z, st, y, layer, unit, blocks, cb, turn, wave, lane, stage1, stage2, stage3);
}

template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads, 2)
attend_kernel(const AttendArgs a) {
  __shared__ u32x4 stage0[kStage], stage1[kStage], stage2[kStage], stage3[kStage];
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
  const Plan p = plan_of<RowsBf16>(a, n, layer, tid);
  // items that fit the chip at once are the longer ones (16 samples of one question: 173 us, shares first 179);
  // items of many rounds end more evenly than shares
  const bool items_first = p.all_items <= (uint32_t)a.both_wgs;
  const uint32_t first_share = items_first ? p.all_items : 0, first_item = items_first ? 0 : p.shares;
  if (id >= first_share && id < first_share + p.shares) {      // uniform
    const int wave = tid >> 6;
    u32x4* tile = wave == 0 ? stage0 : (wave == 1 ? stage1 : (wave == 2 ? stage2 : stage3));
    attend_streams<BF16_OUT>(a, n, p, sh.streams.seg, sh.streams.n_seg, reinterpret_cast<uint16_t*>(tile),
                             id - first_share, layer, tid);
  } else if (id >= first_item && id < first_item + p.all_items) {
    find_item(a, n, p, sh.item.item, id - first_item, tid);
    if (sh.item.item.valid) attend_item<BF16_OUT>(a, n, sh.item, stage0, stage1, stage2, stage3, layer, tid);
  }
}

}  // namespace

// For a call with groups: one without needs no more, in every term.
size_t attend_workspace_bytes(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq) {
  return sizes_of(L, B, n_groups, n_q, Hq / kHeads, can_share(B)).total;
}

hipError_t launch_attend(int32_t L, int32_t B, int32_t n_groups, int32_t n_q, int32_t Hq, const uint16_t* q,
                         const int32_t* q_off, const int32_t* grp_off, const uint16_t* ctx_k, const uint16_t* ctx_v,
                         const int32_t* ctx_len, int32_t max_ctx, const uint16_t* k_pages, const uint16_t* v_pages,
                         int32_t n_pages, int32_t page_shift, const int32_t* page_table, int32_t max_pages,
                         const int32_t* kv_len, const int32_t* pre_len, float scale, bool bf16_out, void* out,
                         void* ws, hipStream_t s) {
  if (!can_share(B)) grp_off = nullptr;      // one sequence, so one group
  const Sizes z = sizes_of(L, B, n_groups, n_q, Hq / kHeads, grp_off != nullptr);
  const AttendArgs a = args_of(z, B, n_groups, n_q, Hq, q, q_off, grp_off, ctx_k, ctx_v, ctx_len, max_ctx, k_pages, v_pages,
                               n_pages, page_shift, page_table, max_pages, kv_len, pre_len, scale, out, ws);
  if (bf16_out) launch_as<RowsBf16, true>(attend_kernel<true>, a, z, L, s);
  else launch_as<RowsBf16, false>(attend_kernel<false>, a, z, L, s);
  return hipGetLastError();
}

}  // namespace msa

