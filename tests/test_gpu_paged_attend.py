"""GPU tests of msa_paged_attend against attention in 64 bits: one token to long prompts, ragged
mixes, groups that share memory rows and local pages, every head group, page sizes that end inside a
tile, rows that are masked or hold no numbers, and the refused calls."""
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


from paged_common import SCALE, Batch, attention, check_attention  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def workspace(b):
    n = msa.msa_paged_attend_workspace_size(b.L, b.B, b.G, b.n_q, b.hq)
    assert n > 0
    return torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)


def attend(b, d=None, dtype=F32, scale=SCALE, fill=7.0, ws=None):
    d = d or b.to_device()
    out = torch.full((b.L, b.n_q, b.hq, 128), fill, dtype=dtype, device="cuda")
    msa.msa_paged_attend(d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], scale, out,
                         workspace(b) if ws is None else ws, grp_off=d["grp_off"], ctx_k=d["ctx_k"],
                         ctx_v=d["ctx_v"], ctx_len=d["ctx_len"], pre_len=d["pre_len"])
    torch.cuda.synchronize()
    assert (out[:, b.q_off[-1]:] == fill).all()      # rows behind the last sequence
    return out


def some(b, n, seed=0):
    """n of the batch's tokens, among them the first and last of every sequence's."""
    rng = np.random.default_rng(seed)
    live = [s for s in range(b.B) if b.new[s]]
    ends = [(l, s, i) for l in (0, b.L - 1) for s in live[:3] + live[-3:] for i in {0, b.new[s] - 1}]
    more = [(int(rng.integers(b.L)), s, int(rng.integers(b.new[s]))) for s in rng.choice(live, n)]
    return ends + more


ONE = [  # new, rows, groups, ctx rows, pre, page
    ([1], [1], None, None, None, 16),
    ([1], [2], None, [1], None, 1),
    ([1], [31], None, [0], None, 16),
    ([1], [33], None, [32], None, 8),
    ([1], [64], None, [100], None, 64),
    ([1, 1, 1], [1, 129, 70], None, [5, 0, 300], None, 32),
    ([1, 0, 1, 1], [40, 3, 1, 200], [4], [77], [32], 16),
    ([1, 1, 0, 0, 1, 1], [70, 90, 64, 0, 65, 66], [2, 1, 3], [10, 0, 33], [64, 0, 0], 32),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hq", [8, 16, 32, 64])
@pytest.mark.parametrize("case", range(len(ONE)))
def test_one_token(case, hq, dtype):
    print("case: one token", case, hq, dtype, flush=True)
    new, rows, groups, ctx, pre, page = ONE[case]
    G = len(groups) if groups else len(new)
    ctx = None if ctx is None else [ctx + [0] * (G - len(ctx)), [c // 2 for c in ctx] + [3] * (G - len(ctx))]
    b = Batch(new, rows, groups=groups, ctx=ctx, pre=pre, page=page, hq=hq, layers=2 if ctx else 1, pad=case % 2,
              seed=100 + case, q_std=2.0)
    check_attention(b, attend(b, dtype=dtype))


MANY = [  # new, rows, groups, ctx rows (one layer), pre, page, hq
    ([2, 5, 9], [2, 30, 100], None, [0, 40, 7], None, 16, 32),
    ([33], [33], None, None, None, 64, 32),
    ([70], [100], None, [50], None, 16, 32),
    ([131], [131], None, [1], None, 128, 8),
    ([40], [333], None, [65], None, 4, 64),
    ([200, 1, 0, 17], [260, 90, 4, 17], None, [33, 0, 5, 64], None, 32, 32),
    ([1] * 9, [65 + s for s in range(9)], [9], [130], [64], 32, 32),
    ([1] * 40, [200 + 3 * s for s in range(40)], [40], [70], [192], 64, 32),
    ([3, 2, 1, 4] * 5, [100] * 20, [20], [0], [96], 16, 64),
    ([1, 100, 1, 1, 60, 1], [130, 228, 129, 140, 188, 131], [4, 2], [200, 31], [128, 100], 64, 32),
    ([300], [300], None, [90], None, 256, 16),
    ([150, 140], [150 + 64, 140 + 64], [2], [257], [64], 64, 32),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_tokens(case, dtype):
    print("case: many tokens", case, dtype, flush=True)
    new, rows, groups, ctx, pre, page, hq = MANY[case]
    b = Batch(new, rows, groups=groups, ctx=None if ctx is None else [ctx], pre=pre, page=page, hq=hq, pad=case % 3,
              seed=200 + case, q_std=2.0)
    check_attention(b, attend(b, dtype=dtype))


def test_tokens_that_see_no_row_are_zero():
    """Fewer local rows than tokens and no memory: the first tokens see nothing; a sequence with none at
    all; and the same behind a shared context of no rows."""
    print("case: no rows", flush=True)
    for groups, pre in ((None, None), ([1, 2], [0, 0]), ([3], [4])):
        b = Batch([8, 2, 1], [5, 2, 7], groups=groups, ctx=[[0] * (len(groups) if groups else 3)], pre=pre, page=4,
                  hq=32, seed=31)
        if groups == [3]:
            b.table[1:, 0] = b.table[0, 0]
        b.rows[1] = 0
        for dtype in (F32, BF16):
            out = attend(b, dtype=dtype)
            assert (out[0, :3] == 0).all() and (out[0, 8:10] == 0).all()
            check_attention(b, out)


def test_pre_len_beyond_a_sequences_rows():
    """Shared rows that some sequences' tokens do not all see: each token's own limit decides."""
    print("case: pre_len beyond rows", flush=True)
    b = Batch([1, 3, 1, 1], [100, 40, 96, 20], groups=[4], ctx=[[17]], pre=[96], page=16, hq=32, seed=41)
    check_attention(b, attend(b))


def test_two_layers_with_different_memory_lengths():
    print("case: layers", flush=True)
    b = Batch([1, 20, 1, 2], [50, 70, 33, 600], groups=[2, 2], ctx=[[0, 400], [333, 1], [64, 0]], pre=[32, 0], page=16,
              hq=32, layers=3, seed=51, q_std=2.0)
    check_attention(b, attend(b))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_are_split_and_joined(dtype):
    print("case: long rows", dtype, flush=True)
    b = Batch([1, 1], [9001, 30], ctx=[[5003, 17], [1, 4999]], page=32, hq=32, layers=2, seed=61, q_std=2.0)
    check_attention(b, attend(b, dtype=dtype))


def test_long_shared_prefix():
    print("case: long shared prefix", flush=True)
    B = 37
    b = Batch([1] * B, [8192 + 1 + 13 * s for s in range(B)], groups=[B], ctx=[[1000]], pre=[8192], page=128, hq=64,
              seed=71, q_std=2.0)
    check_attention(b, attend(b, dtype=BF16), tokens=some(b, 12))
    check_attention(b, attend(b), tokens=some(b, 12))


def test_long_prompt():
    print("case: long prompt", flush=True)
    b = Batch([2500, 1], [2700, 900], ctx=[[700, 100]], page=64, hq=32, seed=81, q_std=2.0)
    check_attention(b, attend(b, dtype=BF16), tokens=some(b, 40))
    check_attention(b, attend(b), tokens=some(b, 40))


def test_many_sequences():
    print("case: 2048 sequences", flush=True)
    rng = np.random.default_rng(5)
    new = rng.choice([0, 1, 1, 1, 2], 2048).tolist()
    rows = [n + int(rng.integers(0, 40)) for n in new]
    groups = []
    while sum(groups) < 2048:
        groups.append(min(int(rng.integers(0, 9)), 2048 - sum(groups)))
    b = Batch(new, rows, groups=groups, ctx=[rng.integers(0, 20, len(groups)).tolist()], page=8, hq=8, seed=91)
    check_attention(b, attend(b), tokens=some(b, 150))
    b = Batch(new, rows, ctx=None, page=8, hq=8, seed=92)
    check_attention(b, attend(b), tokens=some(b, 150))


@pytest.mark.parametrize("groups,pre", [([7], [64]), ([3, 4], [32, 0]), ([1, 5, 1], [0, 64, 9])])
def test_long_sequences_among_short_ones_of_a_group(groups, pre):
    """One at the border (512 columns) and some past it, which read their group's rows themselves."""
    print("case: long sequences in groups", groups, flush=True)
    new = [1, 200, 1, 1, 130, 129, 128]
    ctx = [[100, 33, 70][:len(groups)]]
    b = Batch(new, [n + 70 + s for s, n in enumerate(new)], groups=groups, ctx=ctx, pre=pre, page=32, hq=32, pad=2,
              seed=95, q_std=2.0)
    check_attention(b, attend(b), tokens=some(b, 40))
    check_attention(b, attend(b, dtype=BF16), tokens=some(b, 40))


@pytest.mark.parametrize("groups", [None, 7])
def test_many_short_sequences_in_many_layers(groups):
    """More pieces in a workgroup's share of the rows than it lists at a time."""
    print("case: short sequences, many layers", groups, flush=True)
    rng = np.random.default_rng(17)
    new = rng.choice([0, 1, 1, 2], 700).tolist()
    rows = [n + int(rng.integers(0, 70)) for n in new]
    if groups:
        b = Batch(new, rows, groups=[groups] * 100, ctx=rng.integers(0, 40, (24, 100)).tolist(), page=16, hq=8, layers=24,
                  seed=96)
    else:
        b = Batch(new, rows, page=16, hq=8, layers=24, seed=97)
    check_attention(b, attend(b), tokens=some(b, 150))


def test_many_prompts():
    """2,048 prompts of 64 tokens and 64 query heads: more workgroups than one dimension of a launch holds."""
    print("case: 2048 prompts", flush=True)
    b = Batch([64] * 2048, [64 + s % 3 for s in range(2048)], page=64, hq=64, seed=98)
    check_attention(b, attend(b, dtype=BF16), tokens=some(b, 60))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.3e38])
def test_rows_out_of_sight_do_not_reach_the_output(bad, dtype):
    """Not-a-number, infinite and largest values in every row that no token sees, and, token by token, in
    the rows of the tokens behind it."""
    print("case: bad values in masked rows", bad, dtype, flush=True)
    b = Batch([1, 37, 3, 0, 1, 1, 150], [20, 60, 3, 4, 130, 129, 150], groups=[1, 1, 1, 1, 2, 1],
              ctx=[[9, 33, 0, 4, 65, 70]], pre=[0, 0, 0, 0, 128, 0], page=16, hq=32, seed=101, max_ctx=80)
    clean_k, clean_v, ck, cv = (t.clone() for t in (b.k_pages, b.v_pages, b.ctx_k, b.ctx_v))
    seen = torch.zeros(b.n_pages, b.page, dtype=torch.bool)
    for s in range(b.B):
        for r in range(b.rows[s]):
            seen[b.spot(s, r)] = True
    for pages in (b.k_pages, b.v_pages):
        pages[0][~seen] = bad
    for g, c in enumerate(b.ctx[0]):
        b.ctx_k[0, g, c:] = bad
        b.ctx_v[0, g, c:] = bad
    out = attend(b, dtype=dtype)
    b.ctx_k, b.ctx_v = ck, cv
    check_attention(b, out, k_pages=clean_k, v_pages=clean_v)
    # the last row of each long sequence: all tokens but the last are as they were
    d = b.to_device()
    for s in (1, 2, 6):
        pg, rw = b.spot(s, b.rows[s] - 1)
        d["k_pages"][0, pg, rw] = bad
        d["v_pages"][0, pg, rw] = bad
    d["k_pages"][0][~seen], d["v_pages"][0][~seen] = bad, bad
    out = attend(b, d, dtype=dtype)
    hidden = [(0, s, i) for s in (1, 2, 6) for i in range(b.new[s] - 1)]
    check_attention(b, out, tokens=hidden + [(0, 0, 0), (0, 4, 0), (0, 5, 0)], k_pages=clean_k, v_pages=clean_v)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_seen_does_reach_the_output(value):
    """A V entry that is no finite number comes out in its column of every token that sees it (and of no other)."""
    print("case: visible special value", value, flush=True)
    b = Batch([40, 1], [50, 90], ctx=[[12, 0]], page=16, hq=32, seed=111)
    pg, rw = b.spot(0, 30)                        # seen by tokens 20 .. 39 of sequence 0
    b.v_pages[0, pg, rw, 2, 77] = value
    out = attend(b)
    x = out[0, :40, 8:12, 77]                     # query heads 8 .. 11 read KV head 2
    same = torch.isnan(x) if value != value else x == value
    assert same[20:].all() and torch.isfinite(x[:20]).all()
    out[0, 20:40, 8:12, 77] = 0
    assert torch.isfinite(out).all()


def test_large_scores():
    """Scores of several hundred: one row takes all the weight, nothing overflows."""
    print("case: large scores", flush=True)
    b = Batch([1, 60], [300, 200], ctx=[[40, 0]], page=16, hq=32, seed=121, q_std=40.0)
    for dtype in (F32, BF16):
        check_attention(b, attend(b, dtype=dtype))
    b = Batch([1, 60], [300, 200], ctx=[[40, 0]], page=16, hq=32, seed=122)
    for scale in (1e-6, 0.5, 3.0):
        check_attention(b, attend(b, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_in_the_billions(sign, dtype):
    """Each more than 2^27 from the next (in log2 units): the output is the V row of the largest score."""
    print("case: scores in the billions", sign, dtype, flush=True)
    new, rows = [1, 10, 40], [200, 150, 170]
    b = Batch(new, rows, page=16, hq=32, seed=123)
    rng = np.random.default_rng(123)
    b.q.zero_()
    b.q[..., 0] = 2.0 ** 20
    order = []
    for s in range(3):
        steps = rng.permutation(256)[:rows[s]] + 1
        order.append(steps)
        for r in range(rows[s]):
            pg, rw = b.spot(s, r)
            b.k_pages[0, pg, rw] = 0
            b.k_pages[0, pg, rw, :, 0] = float(sign * steps[r]) * 2.0 ** 12
    out = attend(b, dtype=dtype).cpu()
    for s in range(3):
        for i in range(new[s]):
            r = int(np.argmax(sign * order[s][:rows[s] - new[s] + i + 1]))
            pg, rw = b.spot(s, r)
            v = b.v_pages[0, pg, rw].repeat_interleave(4, 0)
            assert torch.equal(out[0, b.q_off[s] + i], v.to(dtype)), (s, i)


def test_values_near_the_largest():
    """A row that the running maximum, not yet raised, gives a weight of 2^7, with values near the largest."""
    print("case: values near the largest", flush=True)
    new, rows = [1, 10, 40], [100, 100, 100]
    b = Batch(new, rows, page=16, hq=32, seed=124)
    b.q.zero_()
    b.q[..., 0] = 1.0
    for s in range(3):
        for r in range(rows[s]):
            pg, rw = b.spot(s, r)
            b.k_pages[0, pg, rw, :, 0] = 55.0 if r == 40 else 0.0       # 7.01 / (scale log2 e)
            if r == 40:
                b.v_pages[0, pg, rw] = 2.9e38
    for dtype in (F32, BF16):
        check_attention(b, attend(b, dtype=dtype))


def test_rising_scores_move_the_maximum():
    """Keys ordered so that the running maximum rises with almost every tile."""
    print("case: rising scores", flush=True)
    b = Batch([1, 5], [800, 700], page=16, hq=8, seed=131)
    for s in range(2):
        for r in range(b.rows[s]):
            pg, rw = b.spot(s, r)
            b.k_pages[0, pg, rw] = (b.q[0, b.q_off[s]].float() * (r / b.rows[s] * 4)).to(BF16)
    check_attention(b, attend(b))


def test_pages_outside_the_pool_harm_no_other_sequence():
    """Page numbers outside the pool are clamped: reads stay inside it, the other sequences are right."""
    print("case: bad page numbers", flush=True)
    b = Batch([1, 1, 30], [40, 50, 60], ctx=[[5, 6, 7]], page=16, hq=32, seed=141)
    d = b.to_device()
    d["page_table"][1, 0], d["page_table"][1, 1] = -1, 1 << 30
    out = attend(b, d)
    check_attention(b, out, tokens=[(0, 0, 0)] + [(0, 2, i) for i in range(30)])


def test_lengths_past_the_arrays_are_clamped():
    print("case: lengths clamped", flush=True)
    b = Batch([1, 1], [64, 40], ctx=[[10, 20]], page=16, hq=32, seed=151)
    d = b.to_device()
    d["ctx_len"] = b.i32([[-3, 999]])
    d["kv_len"] = b.i32([1 << 30, -7])
    out = attend(b, d)
    b.ctx, b.rows = [[0, 20]], [64, 0]
    b.new = [1, 1]
    ref0, tol0 = attention(b, 0, 0, 0)
    assert ((out[0, 0].cpu().double() - ref0).abs() <= tol0).all()
    ref1, tol1 = attention(b, 0, 1, 0)
    assert ((out[0, 1].cpu().double() - ref1).abs() <= tol1).all()


def test_cache_beyond_32_bit_offsets():
    """Rows in the last pages of a pool of more than 2^31 elements, memory rows of the last group, layer 2."""
    print("case: big offsets", flush=True)
    b = Batch([1, 40], [90, 70], ctx=[[20, 33], [5, 64]], page=64, hq=32, layers=2, seed=161)
    d = b.to_device()
    n_pages = 25000
    shift = n_pages - b.n_pages
    for name in ("k_pages", "v_pages"):
        big = torch.zeros(2, n_pages, 64, 8, 128, dtype=BF16, device="cuda")
        big[:, shift:] = d[name]
        d[name] = big
    d["page_table"] = d["page_table"] + shift
    check_attention(b, attend(b, d))


def test_results_do_not_depend_on_the_neighbours_or_the_run():
    """Two runs give the same bits, whatever the workspace held; sharing changes no value beyond its bound."""
    print("case: determinism", flush=True)
    b = Batch([1] * 12 + [90], [300 + s for s in range(12)] + [350], groups=[12, 1], ctx=[[500, 60]], pre=[256, 0],
              page=64, hq=32, seed=171)
    d = b.to_device()
    for dtype in (F32, BF16):
        x = attend(b, d, dtype=dtype)
        ws = workspace(b).fill_(0x3C)
        y = attend(b, d, dtype=dtype, ws=ws)
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    alone = Batch([1] * 12 + [90], [300 + s for s in range(12)] + [350], page=64, hq=32, seed=171)
    alone.ctx, alone.max_ctx = [[500] * 12 + [60]], 500
    alone.table, alone.n_pages, alone.max_pages = b.table, b.n_pages, b.max_pages
    alone.q, alone.k_pages, alone.v_pages = b.q, b.k_pages, b.v_pages
    alone.ctx_k = torch.stack([b.ctx_k[0, g] for g in b.group_of])[None]
    alone.ctx_v = torch.stack([b.ctx_v[0, g] for g in b.group_of])[None]
    check_attention(alone, attend(alone))


def test_same_as_the_sparse_calls():
    """Against msa_sparse_decode and msa_sparse_prefill on the same rows."""
    print("case: against decode and prefill", flush=True)
    for T in (1, 50):
        L, B, hq, P = 2, 3, 32, 16
        rows, ctx = [T + 30, T, T + 7], [[40, 0, 9], [3, 64, 1]]
        b = Batch([T] * B, rows, ctx=ctx, page=P, hq=hq, layers=L, seed=181 + T)
        got = attend(b)
        d = b.to_device()
        max_loc = max(rows)
        lk = torch.zeros(L, B, max_loc, 8, 128, dtype=BF16)
        lv = torch.zeros_like(lk)
        for l in range(L):
            for s in range(B):
                lk[l, s, :rows[s]] = b.local(b.k_pages, l, s, rows[s])
                lv[l, s, :rows[s]] = b.local(b.v_pages, l, s, rows[s])
        lk, lv = lk.cuda(), lv.cuda()
        ll = torch.tensor([rows] * L, dtype=torch.int32, device="cuda")
        q = d["q"].view(L, B, T, hq, 128)
        if T == 1:
            out = torch.empty(L, B, hq, 128, dtype=F32, device="cuda")
            ws = torch.empty(msa.msa_sparse_decode_workspace_size(L, B, hq, b.max_ctx, max_loc), dtype=torch.uint8,
                             device="cuda")
            msa.msa_sparse_decode(q[:, :, 0].contiguous(), d["ctx_k"], d["ctx_v"], d["ctx_len"], lk, lv, ll, SCALE, out, ws)
        else:
            out = torch.empty(L, B, T, hq, 128, dtype=F32, device="cuda")
            msa.msa_sparse_prefill(q, d["ctx_k"], d["ctx_v"], d["ctx_len"], lk, lv, ll, SCALE, out)
        torch.cuda.synchronize()
        # both are within the bound of the same exact value
        for l in range(L):
            for s in range(B):
                for i in range(T):
                    tol = attention(b, l, s, i)[1]
                    x, y = got[l, b.q_off[s] + i].cpu().double(), (out[l, s] if T == 1 else out[l, s, i]).cpu().double()
                    assert ((x - y).abs() <= 2 * tol).all()


def test_no_tokens():
    b = Batch([0, 0], [3, 4], page=4, hq=8, seed=1, pad=2)
    attend(b)
    b = Batch([0], [3], page=4, hq=8, seed=1)
    attend(b)
