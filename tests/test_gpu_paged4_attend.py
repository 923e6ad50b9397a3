"""GPU tests of msa_paged_attend4 against attention in 64 bits over the values that the pages stand for: the batches
that msa_paged_attend is tested with, tiles that end inside pages and pages inside tiles, rows that are masked or
stand for no numbers, large scores, guarded buffers, streams and graphs, and the serving loop."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from routed_kv_memory_amd import msa
    msa.lib()
    yield
    torch.cuda.synchronize()


import test_gpu_paged_attend as bf16_tests  # noqa: E402
import test_gpu_paged_canaries as canaries  # noqa: E402
import test_gpu_paged_groups as group_tests  # noqa: E402
from paged4_common import ROW4, Batch4, check_every_token, pack, unpack  # noqa: E402
from paged_common import EPS, SCALE, THETA  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
GUARD = 1 << 16


def attend(b, d=None, dtype=F32, scale=SCALE, fill=7.0, ws_fill=0xFF, grp_off=None):
    """The call in a workspace of just its size; nothing around it and no row behind the last sequence changes."""
    d = d or b.to_device()
    size = msa.msa_paged_attend4_workspace_size(b.L, b.B, b.G, b.n_q, b.hq)
    ws = torch.full((size + GUARD,), ws_fill, dtype=torch.uint8, device="cuda")
    out = torch.full((b.L, b.n_q, b.hq, 128), fill, dtype=dtype, device="cuda")
    msa.msa_paged_attend4(d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], scale, out,
                          ws[:size], grp_off=d["grp_off"] if grp_off is None else grp_off, ctx_k=d["ctx_k"],
                          ctx_v=d["ctx_v"], ctx_len=d["ctx_len"], pre_len=d["pre_len"])
    torch.cuda.synchronize()
    assert (ws[size:] == ws_fill).all() and (out[:, b.q_off[-1]:] == fill).all()
    return out


def check(b, out, scale=SCALE):
    """Every token of a batch against 64 bits over the values that its pages stand for."""
    dev = out.device
    ctx = None if b.ctx is None else (b.ctx_k.to(dev), b.ctx_v.to(dev), b.ctx, b.group_of)
    n = b.q_off[-1]
    check_every_token(out[:, :n], b.q[:, :n].to(dev), b.q_off, b.rows, torch.from_numpy(b.table).to(dev),
                      b.k_pages.to(dev), b.v_pages.to(dev), ctx, scale=scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hq", [8, 16, 32, 64])
@pytest.mark.parametrize("case", range(len(bf16_tests.ONE)))
def test_one_token(case, hq, dtype):
    print("case: one token", case, hq, dtype, flush=True)
    new, rows, groups, ctx, pre, page = bf16_tests.ONE[case]
    G = len(groups) if groups else len(new)
    ctx = None if ctx is None else [ctx + [0] * (G - len(ctx)), [c // 2 for c in ctx] + [3] * (G - len(ctx))]
    b = Batch4(new, rows, groups=groups, ctx=ctx, pre=pre, page=page, hq=hq, layers=2 if ctx else 1, pad=case % 2,
               seed=100 + case, q_std=2.0)
    check(b, attend(b, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(bf16_tests.MANY)))
def test_many_tokens(case, dtype):
    print("case: many tokens", case, dtype, flush=True)
    new, rows, groups, ctx, pre, page, hq = bf16_tests.MANY[case]
    b = Batch4(new, rows, groups=groups, ctx=None if ctx is None else [ctx], pre=pre, page=page, hq=hq, pad=case % 3,
               seed=200 + case, q_std=2.0)
    check(b, attend(b, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(group_tests.CASES)))
def test_as_many_groups_as_sequences(case, dtype):
    print("case: groups", case, dtype, flush=True)
    new, rows, groups, pre, hq = group_tests.CASES[case]
    lens = [[(37 * g + 61 * l + 11 * case) % 130 for g in range(len(groups))] for l in range(2)]
    b = Batch4(new, rows, groups=groups, ctx=lens, pre=pre, page=16, hq=hq, layers=2, pad=case % 3, seed=500 + case, q_std=2.0)
    check(b, attend(b, dtype=dtype, grp_off=b.i32(b.grp_off)))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 128, 1024])
@pytest.mark.parametrize("rows", [127, 128, 129, 160, 161, 255, 257, 700])
def test_ends_of_tiles_and_pages(rows, page):
    """Streamed tiles are 128 rows, used in pieces of 32; one token, drafted ones, a piece of a prompt; a shared part that
    ends inside a page, a tile and a piece."""
    print("case: rows %d, pages of %d" % (rows, page), flush=True)
    b = Batch4([1, 3, 20, 1, 1], [rows, rows + 3, rows + 20, rows + 1, rows + 40], groups=[1, 1, 1, 2],
               ctx=[[0, 31, 33, 5]], pre=[0, 0, 0, (rows - 5) // page * page], page=page, hq=32, seed=700 + rows + page, q_std=2.0)
    for dtype in (F32, BF16):
        check(b, attend(b, dtype=dtype))


@pytest.mark.parametrize("odd", [1, 17, 33, 100])
def test_shared_rows_that_do_not_end_with_a_page(odd):
    """pre_len in the middle of a page that all of a group have: the own rows begin there."""
    print("case: odd shared part", odd, flush=True)
    rows = [odd + 90, odd + 200, odd + 128]
    b = Batch4([1, 2, 150], rows, groups=[3], ctx=[[40]], pre=[-(-odd // 64) * 64], page=64, hq=32, seed=730 + odd)
    b.pre = [odd]
    check(b, attend(b))


@pytest.mark.parametrize("columns", [17, 32, 33, 64, 65, 96, 128, 129, 161, 193, 257])
def test_columns_of_a_shared_job(columns):
    print("case: shared columns", columns, flush=True)
    other = [3, 1, 40]
    b = Batch4([1] * columns + other, [300 + s % 7 for s in range(columns)] + [90, 30, 70], groups=[columns, 3],
               ctx=[[900, 33]], pre=[256, 0], page=64, hq=8, seed=540 + columns, q_std=2.0)
    for dtype in (F32, BF16):
        check(b, attend(b, dtype=dtype))


def test_tokens_that_see_no_row_are_zero():
    print("case: no rows", flush=True)
    for groups, pre in ((None, None), ([1, 2], [0, 0]), ([3], [4])):
        b = Batch4([8, 2, 1], [5, 2, 7], groups=groups, ctx=[[0] * (len(groups) if groups else 3)], pre=pre, page=4,
                   hq=32, seed=31)
        if groups == [3]:
            b.table[1:, 0] = b.table[0, 0]
        b.rows[1] = 0
        for dtype in (F32, BF16):
            out = attend(b, dtype=dtype)
            assert (out[0, :3] == 0).all() and (out[0, 8:10] == 0).all()
            check(b, out)


def test_pre_len_beyond_a_sequences_rows():
    print("case: pre_len beyond rows", flush=True)
    b = Batch4([1, 3, 1, 1], [100, 40, 96, 20], groups=[4], ctx=[[17]], pre=[96], page=16, hq=32, seed=41)
    check(b, attend(b))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_are_split_and_joined(dtype):
    print("case: long rows", dtype, flush=True)
    b = Batch4([1, 1, 4], [20001, 30, 7000], ctx=[[5003, 17, 0], [1, 4999, 300]], page=32, hq=32, layers=2, seed=61, q_std=2.0)
    check(b, attend(b, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_shared_prefix_and_a_prompt(dtype):
    print("case: long shared prefix, prompt", dtype, flush=True)
    B = 21
    b = Batch4([1] * B + [600], [8192 + 1 + 13 * s for s in range(B)] + [3000], groups=[B, 1], ctx=[[1000, 77]], pre=[8192, 0],
               page=128, hq=64, seed=71, q_std=2.0)
    check(b, attend(b, dtype=dtype))


def test_many_sequences():
    print("case: 2048 sequences", flush=True)
    rng = np.random.default_rng(5)
    new = rng.choice([0, 1, 1, 1, 2], 2048).tolist()
    rows = [n + int(rng.integers(0, 200)) for n in new]
    groups = []
    while sum(groups) < 2048:
        groups.append(min(int(rng.integers(0, 9)), 2048 - sum(groups)))
    b = Batch4(new, rows, groups=groups, ctx=[rng.integers(0, 20, len(groups)).tolist()], page=8, hq=8, seed=91)
    check(b, attend(b))
    b = Batch4(new, rows, ctx=None, page=8, hq=8, seed=92)
    check(b, attend(b))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sequences,layers", [(2, 1), (9, 1), (24, 2), (24, 18), (70, 1), (130, 2), (257, 1)])
def test_order_of_items(sequences, layers, dtype):
    """Wide sequences of ragged lengths: fewer items than compute units, one round of them with and without chunks to
    spare, several rounds, more sequences than threads of a plan."""
    print("case: order of items", sequences, layers, dtype, flush=True)
    rng = np.random.default_rng(sequences)
    new = [int(rng.choice([5, 5, 9, 0])) if s else 5 for s in range(sequences)]
    rows = [n + int(rng.integers(0, 3000 if sequences < 30 else 300)) for n in new]
    b = Batch4(new, rows, page=16, hq=64, layers=layers, seed=400 + sequences)
    check(b, attend(b, dtype=dtype))


@pytest.mark.parametrize("layers", [1, 7, 18])
@pytest.mark.parametrize("most", [3, 40, 300])
def test_shares_end_anywhere_in_memory_and_local_rows(most, layers):
    """Short streams of memory rows and local ones, which cost unlike: shares that end with a tile, in one, and with a stream."""
    print("case: shares of memory and local rows", most, layers, flush=True)
    rng = np.random.default_rng(most)
    new = [1] * 45
    rows = [1 + int(rng.integers(0, most)) for _ in new]
    ctx = rng.integers(0, most + 1, (layers, 45)).tolist()
    b = Batch4(new, rows, ctx=ctx, page=16, hq=16, layers=layers, seed=500 + most)
    check(b, attend(b))


@pytest.mark.parametrize("grouped", [False, True])
def test_shares_of_many_pieces(grouped):
    """More pieces in a workgroup's share of the rows than it lists at a time, next to shared tiles."""
    print("case: many pieces", grouped, flush=True)
    rng = np.random.default_rng(17)
    new = [int(rng.choice([17, 60])) if s % 50 == 20 else int(rng.choice([0, 1, 1, 2])) for s in range(700)]
    rows = [n + int(rng.integers(0, 270)) for n in new]
    kw = dict(groups=[7] * 100, ctx=rng.integers(0, 40, (24, 100)).tolist()) if grouped else {}
    b = Batch4(new, rows, page=16, hq=8, layers=24, seed=96, **kw)
    check(b, attend(b))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code,byte", [(7, 255), (15, 254), (7, 252), (0, 255)])
def test_rows_out_of_sight_do_not_reach_the_output(code, byte, dtype):
    """Rows that stand for NaN, infinities (6 * 2^127) and the largest values wherever no token sees them, and, token by token, in
    the rows of the tokens behind it."""
    print("case: bad rows out of sight", code, byte, dtype, flush=True)
    b = Batch4([1, 37, 3, 0, 1, 1, 150], [20, 60, 3, 4, 130, 129, 150], groups=[1, 1, 1, 1, 2, 1],
               ctx=[[9, 33, 0, 4, 65, 70]], pre=[0, 0, 0, 0, 128, 0], page=16, hq=32, seed=101, max_ctx=80)
    seen = torch.zeros(b.n_pages, b.page, dtype=torch.bool)
    for s in range(b.B):
        for r in range(b.rows[s]):
            seen[b.spot(s, r)] = True
    bad = float("nan") if byte == 255 else 3.3e38
    for g, c in enumerate(b.ctx[0]):
        b.ctx_k[0, g, c:], b.ctx_v[0, g, c:] = bad, bad

    def spoil(where):
        d = {}
        for name in ("k_pages4", "v_pages4"):
            codes, scales = (t.clone() for t in unpack(getattr(b, name)))
            codes[0][where], scales[0][where] = code, byte
            d[name[:-1]] = pack(codes, scales).cuda()
        return {**b.to_device(), **d}

    ctx_k, ctx_v = b.ctx_k, b.ctx_v
    clean = lambda t: torch.where(torch.isfinite(t.float()) & (t.float().abs() < 1e38), t, torch.zeros_like(t))
    out = attend(b, spoil(~seen), dtype=dtype)
    b.ctx_k, b.ctx_v = clean(ctx_k), clean(ctx_v)
    check(b, out)
    # the last row of each long sequence: all tokens but the last are as they were
    last = ~seen
    for s in (1, 2, 6):
        last[b.spot(s, b.rows[s] - 1)] = True
    b.ctx_k, b.ctx_v = ctx_k, ctx_v
    spoilt = attend(b, spoil(last), dtype=dtype)
    for s in (1, 2, 6):
        t = b.q_off[s + 1] - 1
        spoilt[:, t] = out[:, t]
    b.ctx_k, b.ctx_v = clean(ctx_k), clean(ctx_v)
    check(b, spoilt)


def test_a_block_without_numbers_that_is_seen_does_reach_the_output():
    print("case: visible NaN block", flush=True)
    b = Batch4([40, 1], [50, 90], ctx=[[12, 0]], page=16, hq=32, seed=111)
    codes, scales = unpack(b.v_pages4)
    pg, rw = b.spot(0, 30)                        # seen by tokens 20 .. 39 of sequence 0
    scales[0, pg, rw, 2, 1] = 255                 # dims 32 .. 63 of KV head 2
    d = b.to_device()
    d["v_pages"] = pack(codes, scales).cuda()
    for dtype in (F32, BF16):
        out = attend(b, d, dtype=dtype)
        x = out[0, :40, 8:12, 32:64]              # query heads 8 .. 11 read KV head 2
        assert torch.isnan(x[20:]).all() and torch.isfinite(x[:20]).all()
        out[0, 20:40, 8:12, 32:64] = 0
        assert torch.isfinite(out).all()


def test_large_scores_and_values():
    print("case: large scores", flush=True)
    b = Batch4([1, 60, 5], [300, 200, 500], ctx=[[40, 0, 9]], page=16, hq=32, seed=121, q_std=40.0)
    for dtype in (F32, BF16):
        check(b, attend(b, dtype=dtype))
    b = Batch4([1, 60], [300, 200], ctx=[[40, 0]], page=16, hq=32, seed=122)
    for scale in (1e-6, 0.5, 3.0):
        check(b, attend(b, scale=scale), scale=scale)
    # blocks of very different sizes, and a row whose values are near the largest
    b = Batch4([1, 10, 40], [100, 100, 100], page=16, hq=32, seed=124)
    b.q.zero_()
    b.q[..., 0] = 1.0
    for s in range(3):
        for r in range(100):
            pg, rw = b.spot(s, r)
            b.k_pages[0, pg, rw, :, 0] = 56.0 if r == 40 else 0.0       # 7.1 / (scale log2 e)
            b.v_pages[0, pg, rw] = (b.v_pages[0, pg, rw].float() * 2.0 ** (r % 20 - 10)).to(BF16)
            if r == 40:
                b.v_pages[0, pg, rw] = 2.5e38
    for name in ("k_pages", "v_pages"):
        b.hold(name, getattr(b, name))
    for dtype in (F32, BF16):
        check(b, attend(b, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_in_the_billions(sign, dtype):
    """Each twice the next (2^27 and more apart in log2 units): the output is the V row of the largest score."""
    print("case: scores in the billions", sign, dtype, flush=True)
    new, rows = [1, 10, 40], [70, 64, 60]
    b = Batch4(new, rows, page=16, hq=32, seed=123)
    rng = np.random.default_rng(123)
    b.q.zero_()
    b.q[..., 0] = 2.0 ** 20
    order = []
    for s in range(3):
        steps = rng.permutation(rows[s])
        order.append(steps)
        for r in range(rows[s]):
            pg, rw = b.spot(s, r)
            b.k_pages[0, pg, rw] = 0
            b.k_pages[0, pg, rw, :, 0] = float(sign * 2.0 ** (12 + int(steps[r])))
    b.hold("k_pages", b.k_pages)
    out = attend(b, dtype=dtype).cpu()
    for s in range(3):
        for i in range(new[s]):
            seen = order[s][:rows[s] - new[s] + i + 1]
            r = int(np.argmax(seen) if sign > 0 else np.argmin(seen))
            pg, rw = b.spot(s, r)
            assert torch.equal(out[0, b.q_off[s] + i], b.v_pages[0, pg, rw].repeat_interleave(4, 0).to(dtype)), (s, i)


def test_rising_scores_move_the_maximum():
    print("case: rising scores", flush=True)
    b = Batch4([1, 5], [800, 700], page=16, hq=8, seed=131)
    for s in range(2):
        for r in range(b.rows[s]):
            pg, rw = b.spot(s, r)
            b.k_pages[0, pg, rw] = (b.q[0, b.q_off[s]].float() * (r / b.rows[s] * 4)).to(BF16)
    b.hold("k_pages", b.k_pages)
    check(b, attend(b))


def test_pages_outside_the_pool_harm_no_other_sequence():
    print("case: bad page numbers", flush=True)
    b = Batch4([1, 1, 30], [40, 50, 60], ctx=[[5, 6, 7]], page=16, hq=32, seed=141)
    d = b.to_device()
    d["page_table"][1, 0], d["page_table"][1, 1] = -1, 1 << 30
    out = attend(b, d)
    good = attend(b)
    out[:, 1] = good[:, 1]
    check(b, out)


def test_lengths_past_the_arrays_are_clamped():
    print("case: lengths clamped", flush=True)
    b = Batch4([1, 1], [64, 40], ctx=[[10, 20]], page=16, hq=32, seed=151)
    d = b.to_device()
    d["ctx_len"], d["kv_len"] = b.i32([[-3, 999]]), b.i32([1 << 30, -7])
    out = attend(b, d)
    b.ctx, b.rows = [[0, 20]], [64, 0]
    check(b, out)


def test_cache_beyond_4_gib():
    """Rows in the last pages of a pool of more than 2^32 bytes a layer."""
    print("case: big offsets", flush=True)
    b = Batch4([1, 40, 5], [90, 70, 400], ctx=[[20, 33, 0], [5, 64, 100]], page=64, hq=32, layers=2, seed=161)
    d = b.to_device()
    n_pages = 125000
    shift = n_pages - b.n_pages
    for name in ("k_pages", "v_pages"):
        big = torch.zeros(2, n_pages, 64 * ROW4, dtype=torch.uint8, device="cuda")
        big[:, shift:] = d[name]
        d[name] = big
    d["page_table"] = d["page_table"] + shift
    check(b, attend(b, d))


@pytest.mark.parametrize("case", range(len(canaries.BATCHES)))
def test_guards_and_any_workspace(case):
    """Nothing outside the buffers changes, and the bits do not depend on what the workspace held."""
    print("case: canaries", case, flush=True)
    a = dict(canaries.BATCHES[case])
    a["ctx"] = a["ctx"] * a.get("layers", 1)
    b = Batch4(pad=case % 3, seed=300 + case, q_std=2.0, **a)
    d = b.to_device()
    guarded = {n: canaries.Guarded(d[n]) for n in ("k_pages", "v_pages", "q")}
    d.update({n: x.t for n, x in guarded.items()})
    for dtype in (F32, BF16):
        outs = [attend(b, d, dtype=dtype, ws_fill=fill) for fill in (0, 1, 0xFF)]
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        check(b, outs[0])
    for name, x in guarded.items():
        x.check(name)
        assert torch.equal(x.t.cpu(), b.q if name == "q" else getattr(b, name + "4"))


def test_captured_call_follows_its_lengths():
    print("case: captured, many sequences", flush=True)
    b = Batch4([1] * 400, [60 + s % 5 for s in range(400)], groups=[8] * 50, ctx=[[40] * 50] * 6, page=16, hq=32, layers=6,
               seed=401)
    d = b.to_device()
    ws = torch.empty(msa.msa_paged_attend4_workspace_size(b.L, b.B, b.G, b.n_q, b.hq), dtype=torch.uint8, device="cuda")
    out, eager = (torch.zeros(b.L, b.n_q, b.hq, 128, device="cuda") for _ in range(2))

    def call(to):
        msa.msa_paged_attend4(d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], SCALE, to, ws,
                              grp_off=d["grp_off"], ctx_k=d["ctx_k"], ctx_v=d["ctx_v"], ctx_len=d["ctx_len"])

    call(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    gen = torch.Generator().manual_seed(401)
    for step in range(4):
        d["kv_len"].copy_(torch.randint(1, 65, (400,), generator=gen, dtype=torch.int32).cuda())
        d["ctx_len"].copy_(torch.randint(0, 41, (6, 50), generator=gen, dtype=torch.int32).cuda())
        ws.fill_(step)
        call(eager)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step


class Server:
    """A cache of two layers in 4 bits for five sequences in two groups, and beside it one in bf16 that holds what the
    first one's rows stand for."""

    def __init__(self, seed=3):
        self.L, self.B, self.P, self.hq, self.G = 2, 5, 16, 32, 2
        self.n_pages, self.max_pages = 80, 12
        self.gen = torch.Generator().manual_seed(seed)
        perm = torch.randperm(self.n_pages, generator=self.gen)[:self.B * self.max_pages].view(self.B, self.max_pages)
        self.table = perm.to(torch.int32).cuda()
        self.pages = [torch.randint(0, 256, (2, self.n_pages, self.P * ROW4), generator=self.gen, dtype=torch.uint8).cuda()
                      for _ in range(2)]
        self.kv_len = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        self.pos = torch.full((self.B,), 16, dtype=torch.int32, device="cuda")
        self.grp = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
        self.ctx = [self.rand(self.L, self.G, 90, 8, 128) for _ in range(2)]
        self.lens = [[70, 90], [13, 0]]
        self.ctx_len = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.w_k, self.w_q = self.rand(self.L, 128), self.rand(self.L, 128)

    def rand(self, *s):
        return torch.randn(*s, generator=self.gen).to(BF16).cuda()

    def inputs(self, new):
        n, off = sum(new), np.concatenate([[0], np.cumsum(new)]).tolist()
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        return {"new": i32(new), "q_off": i32(off), "off": off, "k": self.rand(self.L, n, 8, 128),
                "v": self.rand(self.L, n, 8, 128), "q": self.rand(self.L, n, self.hq, 128),
                "q_out": torch.empty(self.L, n, self.hq, 128, dtype=BF16, device="cuda"),
                "out": torch.empty(self.L, n, self.hq, 128, dtype=F32, device="cuda"),
                "ws": torch.empty(msa.msa_paged_attend4_workspace_size(self.L, self.B, self.G, n, self.hq),
                                  dtype=torch.uint8, device="cuda")}

    def step(self, x):
        self.kv_len += x["new"]
        msa.msa_paged_append4(x["k"], x["v"], x["q"], x["q_off"], self.kv_len, self.table, *self.pages, x["q_out"], EPS,
                              THETA, pos_off=self.pos, w_k=self.w_k, w_q=self.w_q)
        msa.msa_paged_attend4(x["q_out"], x["q_off"], self.kv_len, self.table, *self.pages, SCALE, x["out"], x["ws"],
                              grp_off=self.grp, ctx_k=self.ctx[0], ctx_v=self.ctx[1], ctx_len=self.ctx_len)


def test_serving_loop():
    """Prompts, then tokens: each step's output against 64 bits over the rows that msa_paged_read4 gives back."""
    print("case: serving loop", flush=True)
    sv = Server()
    rows = [0] * sv.B
    for new in ([20, 1, 7, 33, 0], [1, 1, 1, 1, 40], [1, 0, 1, 1, 1], [3, 1, 1, 0, 100], [1, 1, 1, 1, 1]):
        x = sv.inputs(new)
        sv.step(x)
        rows = [r + n for r, n in zip(rows, new)]
        off = np.concatenate([[0], np.cumsum(rows)]).tolist()
        k, v = (torch.empty(sv.L, off[-1], 8, 128, dtype=BF16, device="cuda") for _ in range(2))
        msa.msa_paged_read4(*sv.pages, torch.tensor(off, dtype=torch.int32, device="cuda"), sv.table, k, v)
        torch.cuda.synchronize()
        # as pages of one row: sequence b's row r is page off[b] + r
        table = torch.zeros(sv.B, max(rows), dtype=torch.int32, device="cuda")
        for b in range(sv.B):
            table[b, :rows[b]] = torch.arange(off[b], off[b + 1])
        check_every_token(x["out"], x["q_out"], x["off"], rows, table, k[:, :, None], v[:, :, None],
                          (*sv.ctx, sv.lens, [0, 0, 0, 1, 1]))


def test_captured_step_replays_like_the_eager_one():
    print("case: captured step", flush=True)
    eager, graph = Server(7), Server(7)
    a = eager.inputs([30, 2, 9, 17, 1])
    copy = lambda x: {k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()}
    b = copy(a)
    eager.step(a)
    graph.step(b)
    xe = eager.inputs([1, 1, 0, 1, 1])
    xg = copy(xe)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step(xg)
    for rep in range(4):
        eager.step(xe)
        want = [t.clone() for t in (xe["out"], xe["q_out"], *eager.pages, eager.kv_len)]
        xe["ws"].fill_(0xA5)
        xg["ws"].fill_(0x5A)
        xg["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for u, w in zip((xg["out"], xg["q_out"], *graph.pages, graph.kv_len), want):
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), rep
        for name in ("k", "v", "q"):              # the next token's inputs, at the same addresses
            xe[name].copy_(eager.rand(*xe[name].shape))
            xg[name].copy_(xe[name])


def test_two_streams_and_one_workspace_each():
    print("case: two streams", flush=True)
    alone, both = [Server(11), Server(12)], [Server(11), Server(12)]
    xs = [s.inputs([60, 1, 2, 5, 40]) for s in alone]
    ys = [{k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()} for x in xs]
    for s, x in zip(alone, xs):
        s.step(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, y, st in zip(both, ys, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                s.kv_len.zero_()
                s.step(y)
    torch.cuda.synchronize()
    for s, t, x, y in zip(alone, both, xs, ys):
        assert torch.equal(x["out"], y["out"]) and torch.equal(x["q_out"].view(torch.int16), y["q_out"].view(torch.int16))
        assert torch.equal(s.pages[0], t.pages[0]) and torch.equal(s.pages[1], t.pages[1])
    # the stream that is passed is the one that is used
    z = xs[0]
    want = z["out"].clone()
    z["out"].zero_()
    streams[0].wait_stream(torch.cuda.current_stream())
    s = alone[0]
    msa.msa_paged_attend4(z["q_out"], z["q_off"], s.kv_len, s.table, *s.pages, SCALE, z["out"], z["ws"], grp_off=s.grp,
                          ctx_k=s.ctx[0], ctx_v=s.ctx[1], ctx_len=s.ctx_len, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(z["out"], want)


def test_no_tokens_and_refusals_on_the_gpu():
    b = Batch4([0, 0], [3, 4], page=4, hq=8, seed=1, pad=2)
    attend(b)
    b = Batch4([0], [3], page=4, hq=8, seed=1)
    attend(b)
    b = Batch4([2], [2], page=16, hq=8, seed=15)
    d = b.to_device()
    out = torch.empty(1, 2, 8, 128, device="cuda")
    ws = torch.empty(msa.msa_paged_attend4_workspace_size(1, 1, 1, 2, 8), dtype=torch.uint8, device="cuda")
    good = [d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], SCALE, out, ws]
    for at, bad, error in ((5, d["v_pages"].to(torch.int8), TypeError), (5, d["v_pages"][:, :1].contiguous(), ValueError),
                           (4, b.k_pages.cuda(), ValueError), (7, out.half(), TypeError), (8, ws[:-1], msa.MsaError),
                           (6, -1.0, msa.MsaError), (2, d["kv_len"].cpu(), ValueError),
                           (4, d["k_pages"][..., :-1].contiguous(), ValueError)):
        args = list(good)
        args[at] = bad
        with pytest.raises(error):
            msa.msa_paged_attend4(*args)


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("local", [1, 31, 32, 33, 63, 64, 65, 95, 97, 128, 129])
def test_ends_of_streamed_tiles(local, page):
    """Streamed tiles are 64 local rows, used 32 at a time, or 16 memory rows: one and two tokens that end with, before and
    behind them, and a shared part of as many rows."""
    print("case: ends of streamed tiles, %d rows, pages of %d" % (local, page), flush=True)
    memory = [0, 1, 15, 16, 17, 31, 32, 33]
    new = [1, 2] * 4 + [1, 1]
    rows = [max(n, local) for n in new[:8]] + [local + 65, local + 1]
    b = Batch4(new, rows, groups=[1] * 8 + [2], ctx=[memory + [16]], pre=[0] * 8 + [local // page * page], page=page, hq=64,
               seed=800 + local, q_std=2.0)
    for dtype in (F32, BF16):
        check(b, attend(b, dtype=dtype))
