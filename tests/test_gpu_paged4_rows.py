"""GPU tests of msa_paged_append4 and msa_paged_read4 against the format's definition in 64 bits: every code and
scale byte, borders, extreme and non-finite values, rows that are not there, and the run into memory blocks."""
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


from paged4_common import ROW4, Batch4, pack, quantise, unpack, values  # noqa: E402
from paged_common import EPS, THETA, turned  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

BF16 = torch.bfloat16


def append(b, d, pos=None, norm="kq", q=True, theta=THETA, eps=EPS):
    q_out = torch.full_like(d["q"], 5.0) if q else None
    msa.msa_paged_append4(d["k_new"], d["v_new"], d["q"] if q else None, d["q_off"], d["kv_len"], d["page_table"],
                          d["k_pages"], d["v_pages"], q_out, eps, theta, pos_off=None if pos is None else b.i32(pos),
                          w_k=d["w_k"] if "k" in norm else None, w_q=d["w_q"] if "q" in norm and q else None)
    torch.cuda.synchronize()
    return q_out


def check_pages(b, before, after, want, slack):
    """All bytes of after [L][n_pages][544 P] (numpy-like, on the host): rows in `want` {(layer, seq, local row): (value,
    size)} as the definition has them (a value within `slack` times its size of a border may fall to either
    side), all others as before."""
    codes, scales = unpack(after)
    codes0, scales0 = (t.clone() for t in unpack(before))
    for (l, s, r), (x, size) in want.items():
        page, at = b.spot(s, r)
        ends = [quantise(x - slack * size), quantise(x + slack * size)] if slack else [quantise(x)] * 2
        got = codes[l, page, at].clone(), scales[l, page, at]
        low, high = ((c.int(), e.int()) for c, e in ends)
        if slack:                                  # a sum of two zeros may have either sign
            zero = x == 0
            got[0][zero] &= 7
            for c, _ in (low, high):
                c[zero] &= 7
        sure = (low[1] == high[1])
        assert torch.equal(got[1].int()[sure], low[1][sure]), (l, s, r)
        same = (low[0] == high[0]) & sure.repeat_interleave(32, -1)
        # nearly all of them, and no code further off than the two ends
        assert torch.equal(got[0].int()[same], low[0][same]), (l, s, r)
        assert (~same).sum() <= 8, (l, s, r)
        assert ((got[0] == low[0]) | (got[0] == high[0]))[sure.repeat_interleave(32, -1)].all()
        codes0[l, page, at], scales0[l, page, at] = codes[l, page, at], got[1]
    assert torch.equal(codes, codes0) and torch.equal(scales, scales0)      # nothing else was touched


CASES = [  # new, rows, page, hq, layers, pad, norm, far, q
    ([1], [1], 16, 32, 1, 0, "kq", 0, True),
    ([1], [65], 64, 8, 3, 1, "kq", 7, True),
    ([3, 0, 5], [3, 9, 40], 1, 16, 2, 2, "k", 1000, True),
    ([33, 1, 17], [33, 4, 20], 4, 64, 1, 0, "q", 1 << 16, True),
    ([40, 2], [140, 2], 32, 32, 2, 5, "", 1 << 20, True),
    ([257], [300], 1024, 32, 1, 0, "kq", 1 << 22, True),
    ([7, 9], [7, 11], 8, 32, 2, 3, "k", 3, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case):
    new, rows, page, hq, layers, pad, norm, far, q = CASES[case]
    print("case: append4", CASES[case], flush=True)
    b = Batch4(new, rows, page=page, hq=hq, layers=layers, pad=pad, seed=300 + case)
    d = b.to_device()
    pos = [far + 13 * s for s in range(b.B)] if far else None
    q_out = append(b, d, pos, norm, q)
    want_k, want_v, most = {}, {}, 0
    for l in range(b.L):
        for s in range(b.B):
            for i in range(b.new[s]):
                t, r = b.q_off[s] + i, b.rows[s] - b.new[s] + i
                p = r + (pos[s] if pos else 0)
                most = max(most, p)
                x, size = turned(b.k_new[l, t:t + 1], b.w_k[l] if "k" in norm else None, [p])
                want_k[l, s, r] = x[0], size[0]
                want_v[l, s, r] = b.v_new[l, t].double(), torch.zeros(8, 128)
    # fp64: a frequency is a product of up to 11 factors, off by less than 2^-49; an angle by its size times
    # that on either side; 2^-45 for everything else
    check_pages(b, b.k_pages4, d["k_pages"].cpu(), want_k, 2.0 ** -45 + most * 2.0 ** -48)
    check_pages(b, b.v_pages4, d["v_pages"].cpu(), want_v, 0.0)
    if q:                                          # what the append in bf16 makes of q, to the bit
        ref = torch.full_like(d["q"], 5.0)
        k, v = (torch.zeros(b.L, b.n_pages, page, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
        msa.msa_paged_append(d["k_new"], d["v_new"], d["q"], d["q_off"], d["kv_len"], d["page_table"], k, v, ref, EPS, THETA,
                             pos_off=None if pos is None else b.i32(pos), w_k=d["w_k"] if "k" in norm else None,
                             w_q=d["w_q"] if "q" in norm else None)
        assert torch.equal(q_out, ref)


def test_rows_as_they_are():
    """theta 0, no norm: every kind of block, borders to the bit; q comes back unchanged."""
    print("case: append4 of rows as they are", flush=True)
    b = Batch4([12], [12], page=8, hq=8, layers=1, seed=7)
    x = torch.zeros(12, 8, 128)
    steps = torch.tensor([0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0])
    for row in range(4):                           # borders of all codes, and just beside them
        y = steps * 2.0 ** (9 * row - 12)
        y = torch.cat([y, -y, y * (1 + 2.0 ** -7)])[:32]
        x[row] = y.repeat(4)[None]
    x[4, :, 3] = 7.0                               # one value; 7 * 2^e exactly, and a step of bf16 above it
    x[4, :, 40] = 7.03125
    x[5] = 3.3e38                                  # the largest: cut off
    x[5, :, 64:96] = 2.0 ** -133                   # below the smallest scale
    x[6, :, 5] = float("inf")
    x[6, :, 50] = float("nan")
    x[6, :, 51] = float("-inf")
    x[6, :, 100] = 2.0
    x[7] = -0.0
    x[8:] = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(3)) * 2.0 ** torch.arange(-60, 68, 1.0)
    rows = x.to(BF16)
    b.k_new[0], b.v_new[0] = rows, rows.flip(0)
    d = b.to_device()
    q_out = append(b, d, norm="", theta=0.0)
    assert torch.equal(q_out, d["q"])
    none = torch.zeros(8, 128)
    for name, given in (("k_pages", rows), ("v_pages", rows.flip(0))):
        check_pages(b, getattr(b, name + "4"), d[name].cpu(), {(0, 0, r): (given[r].double(), none) for r in range(12)}, 0.0)
    k, v = (torch.empty(1, 12, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
    msa.msa_paged_read4(d["k_pages"], d["v_pages"], d["q_off"], d["page_table"], k, v)
    want = values(*quantise(rows)).to(BF16)
    same = lambda a, w: bool(((a == w) | (a.isnan() & w.isnan())).all())
    assert same(k[0].cpu(), want) and same(v[0].cpu(), want.flip(0))
    assert v[0].isnan().sum() == 8 * 64 == k[0].isnan().sum()          # the two blocks of each head, no others


@pytest.mark.parametrize("norm", ["", "q"])
@pytest.mark.parametrize("hq", [8, 64])
def test_no_rotation_takes_no_dim_to_another(norm, hq):
    """theta 0 and queries with infinities, NaN and zeros of either sign: without a norm the bits of q, with one each
    dim by itself."""
    print("case: append4 without rotation, odd queries", norm, hq, flush=True)
    b = Batch4([9], [9], page=4, hq=hq, layers=2, seed=16)
    inf, nan = float("inf"), float("nan")
    q = b.q
    q[:, 0] = -0.0
    q[:, 1, :, 3], q[:, 2, :, 70], q[:, 3, :, 5] = inf, -inf, nan
    q[:, 4, :, 9], q[:, 4, :, 73] = inf, -inf               # both of a pair that a rotation would turn
    q[:, 5, :, :64], q[:, 6, :, 64:] = -0.0, -0.0
    q[:, 7] = q[:, 7].abs().neg()
    q[:, 7, :, :64] = -0.0                                  # -0 beside negative partners
    d = b.to_device()
    got = append(b, d, norm=norm, theta=0.0).cpu()
    if not norm:
        assert torch.equal(got.view(torch.int16), q.view(torch.int16))
        return
    x = q.double()
    want = x / torch.sqrt((x * x).mean(-1, keepdim=True) + float(np.float32(EPS))) * b.w_q.double()[:, None, None]
    assert torch.equal(got.isnan(), want.isnan())           # of a head with infinities those alone, with a NaN all
    ok = ~want.isnan()
    assert torch.equal(torch.signbit(got)[ok], torch.signbit(want)[ok])
    # fp32: 16 squares summed in a lane, 3 sums over lanes, mean, eps, root, 1 / it (2 steps each), two products; then bf16
    bound = want.abs() * (2.0 ** -8 + 34 * 2.0 ** -24)
    assert bool(((got.double() - want).abs() <= bound)[ok].all())


def test_norm_and_turn_of_odd_rows():
    """Rows of zeros (the norm's eps alone), very large and very small ones, an infinity and a NaN."""
    print("case: append4 of odd rows", flush=True)
    b = Batch4([6], [9], page=4, hq=8, layers=1, seed=8)
    b.k_new[0, 0] = 0
    b.k_new[0, 1] *= 2.0 ** 60
    b.k_new[0, 2] *= 2.0 ** -60
    b.k_new[0, 3, 2, 7] = float("inf")
    b.k_new[0, 4, 5, 80] = float("nan")
    d = b.to_device()
    append(b, d, [100])
    want = {}
    for i in range(6):
        x, size = turned(b.k_new[0, i:i + 1], b.w_k[0], [103 + i])
        want[0, 0, 3 + i] = x[0], torch.nan_to_num(size[0])
    check_pages(b, b.k_pages4, d["k_pages"].cpu(), want, 2.0 ** -40)
    _, scales = unpack(d["k_pages"].cpu())
    page, at = b.spot(0, 7)
    assert (scales[0, page, at, 5] == 255).all() and (scales[0, page, at, 4] < 255).all()


@pytest.mark.parametrize("up,down", [(120, -20), (125, -30), (100, -28), (-60, 100), (127, 0)])
def test_norm_of_keys_whose_factor_is_below_the_smallest_float(up, down):
    """Large keys with small weights: 1 / rms times a weight is below fp32's normal numbers, the key that it makes is
    not."""
    print("case: append4 of keys times 2^%d, weights times 2^%d" % (up, down), flush=True)
    b = Batch4([40], [40], page=8, hq=8, layers=1, seed=10)
    b.k_new = (b.k_new.float().clamp(-1.9, 1.9) * 2.0 ** up).to(BF16)
    b.w_k = (b.w_k.float() * 2.0 ** down).to(BF16)
    d = b.to_device()
    append(b, d, eps=0.0)
    want = {}
    for i in range(40):
        x, size = turned(b.k_new[0, i:i + 1], b.w_k[0], [i], eps=0.0)
        want[0, 0, i] = x[0], size[0]
    check_pages(b, b.k_pages4, d["k_pages"].cpu(), want, 2.0 ** -40)


def test_rows_without_a_place_are_not_stored():
    """Local rows below 0, past the table and on pages that are none; their q is turned all the same."""
    print("case: append4 without a place", flush=True)
    b = Batch4([4, 3, 2, 2], [2, 40, 2, 30], page=8, hq=16, layers=2, pad=1, seed=9)
    table = b.table.copy()
    table[2, 0], table[3, 3] = b.n_pages, -1
    kv = [2, 8 * b.max_pages + 1, 2, 30]           # two rows below 0; one past the table; a page too far; none
    d = b.to_device()
    d["page_table"], d["kv_len"] = torch.from_numpy(table).cuda(), b.i32(kv)
    q_out = append(b, d)
    assert (q_out[:, b.q_off[-1]:] == 5).all() and not (q_out[:, :b.q_off[-1]] == 5).all(-1).any()
    b.table = table
    want = {}
    for l in range(2):
        for s, i in ((0, 2), (0, 3), (1, 0), (1, 1)):
            r = kv[s] - b.new[s] + i
            x, size = turned(b.k_new[l, b.q_off[s] + i:b.q_off[s] + i + 1], b.w_k[l], [r])
            want[l, s, r] = x[0], size[0]
    check_pages(b, b.k_pages4, d["k_pages"].cpu(), want, 2.0 ** -40)


@pytest.mark.parametrize("page", [1, 2, 8, 64, 512])
@pytest.mark.parametrize("first", [0, 5])
def test_read(page, first):
    """Any bytes: all codes, scale bytes 2 to 252 and 255; ragged rows, some from the middle, padding before and behind."""
    print("case: read4", page, first, flush=True)
    b = Batch4([70, 0, 1, 333], [100, 4, 9, 333], page=page, layers=3, pad=3, seed=11)
    g = torch.Generator().manual_seed(page)
    for name in ("k_pages4", "v_pages4"):
        codes = torch.randint(0, 16, (3, b.n_pages, page, 8, 128), generator=g, dtype=torch.uint8)
        scales = torch.randint(2, 254, (3, b.n_pages, page, 8, 4), generator=g, dtype=torch.uint8)
        scales[scales == 253] = 255
        setattr(b, name, pack(codes, scales))
        setattr(b, name[:-1], values(codes, scales).to(BF16))
    d = b.to_device()
    off = [first + x for x in b.q_off]
    n = off[-1] + 3
    k, v = (torch.full((3, n, 8, 128), 9.0, dtype=BF16, device="cuda") for _ in range(2))
    row0 = [r - w for r, w in zip(b.rows, b.new)]
    msa.msa_paged_read4(d["k_pages"], d["v_pages"], b.i32(off), d["page_table"], k, v, row0=b.i32(row0))
    for got, pages in ((k.cpu(), b.k_pages), (v.cpu(), b.v_pages)):
        want = torch.full_like(got, 9.0)
        for l in range(3):
            for s in range(b.B):
                want[l, off[s]:off[s + 1]] = b.local(pages, l, s, b.rows[s])[row0[s]:]
        assert bool(((got == want) | (got.isnan() & want.isnan())).all())
        assert torch.equal(torch.signbit(got)[~got.isnan()], torch.signbit(want)[~want.isnan()])


def test_read_rows_that_are_not_there():
    print("case: read4 of rows that are not there", flush=True)
    b = Batch4([10, 10, 10], [10, 10, 10], page=4, layers=1, seed=12)
    table = b.table.copy()
    table[1, 1], table[1, 2] = b.n_pages, -5
    d = b.to_device()
    d["page_table"] = torch.from_numpy(table).cuda()
    k, v = (torch.full((1, 30, 8, 128), 9.0, dtype=BF16, device="cuda") for _ in range(2))
    row0 = [-3, 0, 4 * b.max_pages - 2]
    msa.msa_paged_read4(d["k_pages"], d["v_pages"], d["q_off"], d["page_table"], k, v, row0=b.i32(row0))
    for got, pages in ((k.cpu(), b.k_pages), (v.cpu(), b.v_pages)):
        want = torch.zeros_like(got)
        want[0, 3:10] = b.local(pages, 0, 0, 7)
        want[0, 10:14] = b.local(pages, 0, 1, 4)
        page, at = int(table[2, -1]), 2
        want[0, 20:22] = pages[0, page, at:at + 2]
        assert torch.equal(got, want)


def test_pages_past_4_gib():
    """Bytes behind the 32-bit range, in the last layer and page."""
    print("case: pages past 4 GiB", flush=True)
    L, n_pages, page = 2, 70000, 64
    pages = [torch.zeros(L, n_pages, page * ROW4, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(2)
    new = [torch.randn(L, 2, 8, 128, generator=g).to(BF16) for _ in range(2)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, off = i32([[n_pages - 1, n_pages - 2]]), i32([0, 2])
    msa.msa_paged_append4(new[0].cuda(), new[1].cuda(), None, off, i32([65]), table, *pages, None, EPS, 0.0)
    out = [torch.empty(L, 2, 8, 128, dtype=BF16, device="cuda") for _ in range(2)]
    msa.msa_paged_read4(*pages, off, table, *out, row0=i32([63]))
    for x, y in zip(new, out):
        assert torch.equal(y.cpu(), values(*quantise(x)).to(BF16))
    assert int(pages[0][:, :n_pages - 2].max()) == 0


def test_ended_sequences_become_memory_blocks():
    """append4, read4, msa_pool_blocks, msa_gather_ctx's input: the pooled rows are the means of the values held."""
    print("case: append4, read4, pool", flush=True)
    new = [130, 64, 1, 75]
    b = Batch4(new, new, page=16, hq=8, layers=2, seed=13)
    d = b.to_device()
    append(b, d)
    k, v = (torch.empty(2, b.n_q, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
    msa.msa_paged_read4(d["k_pages"], d["v_pages"], d["q_off"], d["page_table"], k, v)
    tok = np.asarray(b.q_off, np.int64)
    blk, n_blk, _ = msa.msa_block_offsets_host(tok)
    kb, vb = (torch.empty(2, n_blk, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
    krt = torch.empty(2, msa.msa_route_tiles(n_blk) * 16, 8, 128, dtype=BF16, device="cuda")
    msa.msa_pool_blocks(k, v, k, torch.from_numpy(tok).cuda(), blk.cuda(), n_blk, kb, vb, krt)
    torch.cuda.synchronize()
    at = 0
    for s, n in enumerate(new):
        rows = b.v_new[:, b.q_off[s]:b.q_off[s + 1]]
        held = values(*quantise(rows))
        for lo in range(0, n, 64):
            mean = held[:, lo:lo + 64].mean(1).to(BF16)
            assert torch.equal(vb[:, at].cpu(), mean), (s, lo)
            at += 1
    assert at == n_blk


def test_calls_on_another_stream_and_in_a_graph():
    """append4 and read4 on a stream of their own and replayed: the same bytes as the eager call's."""
    print("case: append4 and read4, stream and graph", flush=True)
    b = Batch4([5, 0, 9], [50, 3, 9], page=16, hq=32, layers=2, seed=14)
    d = b.to_device()
    first = append(b, d)
    k, v = (torch.empty(2, b.n_q, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
    row0 = b.i32([r - n for r, n in zip(b.rows, b.new)])
    msa.msa_paged_read4(d["k_pages"], d["v_pages"], d["q_off"], d["page_table"], k, v, row0=row0)
    e = b.to_device()
    q_out, k2, v2 = torch.zeros_like(first), torch.zeros_like(k), torch.zeros_like(v)

    def both(stream=None):
        msa.msa_paged_append4(e["k_new"], e["v_new"], e["q"], e["q_off"], e["kv_len"], e["page_table"], e["k_pages"],
                              e["v_pages"], q_out, EPS, THETA, w_k=e["w_k"], w_q=e["w_q"], stream=stream)
        msa.msa_paged_read4(e["k_pages"], e["v_pages"], e["q_off"], e["page_table"], k2, v2, row0=row0, stream=stream)

    def same():
        torch.cuda.synchronize()
        n = b.q_off[-1]
        assert torch.equal(k2[:, :n], k[:, :n]) and torch.equal(v2[:, :n], v[:, :n])
        assert torch.equal(q_out[:, :n], first[:, :n]) and torch.equal(e["k_pages"], d["k_pages"])

    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    both(other)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        e["k_pages"].copy_(b.k_pages4)
        e["v_pages"].copy_(b.v_pages4)
        for t in (q_out, k2, v2):
            t.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        same()


def test_refusals_on_the_gpu():
    b = Batch4([2], [2], page=16, hq=8, seed=15)
    d = b.to_device()
    args = [d["k_new"], d["v_new"], d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"],
            torch.empty_like(d["q"]), EPS, THETA]
    for at, bad, error in ((7, d["v_pages"].to(torch.int8), TypeError), (7, d["v_pages"][:, :1].contiguous(), ValueError),
                           (4, d["kv_len"].long(), TypeError), (3, d["q_off"].cpu(), ValueError),
                           (6, d["k_pages"][:, :, :7 * ROW4].contiguous(), ValueError), (10, -1.0, msa.MsaError),
                           (6, torch.empty(1, b.n_pages, 7 * ROW4, dtype=torch.uint8, device="cuda"), ValueError)):
        bads = list(args)
        bads[at] = bad
        with pytest.raises(error):
            msa.msa_paged_append4(*bads)
    seven = torch.empty(1, b.n_pages, 7 * ROW4, dtype=torch.uint8, device="cuda")
    with pytest.raises(msa.MsaError, match="page_tokens=7"):
        msa.msa_paged_read4(seven, seven, d["q_off"], d["page_table"], d["k_new"], d["v_new"])
    with pytest.raises(ValueError, match="v_out"):
        msa.msa_paged_read4(d["k_pages"], d["v_pages"], d["q_off"], d["page_table"], d["k_new"], d["v_new"][:, :1].contiguous())


NEAR = 2.0 ** -40


def candidates(n, positions, norm, turn, w, gen):
    """Heads whose codes or scale bytes come out otherwise in fp32 than in 64 bits: of each position, among n random heads, up to 8
    [8][128] bf16, those with another scale byte first (filled up with any others), how many they are, and how many of
    them have another scale byte."""
    f = torch.tensor([THETA ** (-e / 64.0) for e in range(64)], dtype=torch.float64).cuda()
    w = w.cuda()
    elements = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]).cuda()

    def exponent(x):                              # exact in either width
        m = x.unflatten(-1, (4, 32)).abs().amax(-1)
        mant, e = torch.frexp(m)                  # m = mant 2^e, mant in [0.5, 1)
        return e - 3 + (mant > 0.875).int()

    def codes(x):
        y = torch.ldexp(x.unflatten(-1, (4, 32)).abs(), -exponent(x)[..., None]).flatten(-2)
        c = torch.zeros_like(y, dtype=torch.int32)
        for i, v in enumerate(elements.tolist()):
            c += (y >= v) if i % 2 else (y > v)
        return c

    for p in positions:
        x = torch.randn(n, 128, generator=gen, device="cuda").to(BF16)
        x64, x32 = x.double(), x.float()
        if norm:
            inv = 1.0 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + float(np.float32(EPS)))
            x64, x32 = x64 * (inv * w.double()), x32 * (inv.float() * w.float())
        if turn:
            part = p * f / (2 * np.pi)
            half = 2.0 * (part - torch.round(part))
            pair = lambda y, c, s: torch.cat([y[:, :64] * c - y[:, 64:] * s, y[:, 64:] * c + y[:, :64] * s], 1)
            x64 = pair(x64, torch.cos(np.pi * half), torch.sin(np.pi * half))
            half = half.float().double()
            x32 = pair(x32, torch.cos(np.pi * half).float(), torch.sin(np.pi * half).float())
        other = (exponent(x64) != exponent(x32)).any(-1)
        any_other = other | (codes(x64) != codes(x32)).any(-1)
        rank = any_other.int() + other.int()
        best, at = rank.sort(descending=True, stable=True)
        yield x[at[:8]], int((best[:8] > 0).sum()), int((best[:8] > 1).sum())


@pytest.mark.parametrize("norm,turn,n,least", [(True, True, 1 << 17, 200), (False, True, 1 << 17, 200), (True, False, 1 << 17, 100)])
def test_codes_that_fp32_leaves_open(norm, turn, n, least):
    """Keys next to borders of two codes or exponents, where arithmetic in fp32 falls to the other side: the bytes are those of 64
    bits.  Every value is exact, or further from a border than 64 bits leave open (positions are below 256), so all bytes
    count."""
    print("case: append4, codes that fp32 leaves open", norm, turn, flush=True)
    T = 256
    b = Batch4([T], [T], page=16, hq=8, layers=1, seed=17)
    gen = torch.Generator(device="cuda").manual_seed(17 + 2 * norm + turn)
    found = scales = 0
    for t, (rows, many, of_scales) in enumerate(candidates(n, range(T), norm, turn, b.w_k[0], gen)):
        b.k_new[0, t] = rows.cpu()
        found, scales = found + many, scales + of_scales
    print("heads that differ in fp32: %d of %d, in a scale byte: %d" % (found, 8 * T, scales), flush=True)
    assert found >= least and scales >= 1
    w = b.w_k[0] if norm else None
    want = {}
    for t in range(T):
        x, size = turned(b.k_new[0, t:t + 1], w, [t]) if turn else (b.k_new[0, t:t + 1].double(), None)
        if not turn:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + float(np.float32(EPS))) * w.double()
            size = x.abs()
        ends = quantise(x[0] - NEAR * size[0]), quantise(x[0] + NEAR * size[0])
        exact = not norm and t == 0               # cosines of 1 and sines of 0: the keys as they are, on borders too
        assert exact and torch.equal(x[0], b.k_new[0, t].double()) or torch.equal(ends[0][0], ends[1][0]) and torch.equal(ends[0][1], ends[1][1])
        want[0, 0, t] = x[0], size[0]
    d = b.to_device()
    append(b, d, norm="k" if norm else "", q=False, theta=THETA if turn else 0.0)
    check_pages(b, b.k_pages4, d["k_pages"].cpu(), want, 0.0)
