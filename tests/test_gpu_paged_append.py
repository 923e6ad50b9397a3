"""GPU tests of msa_paged_append against the formulas in 64 bits: ragged batches with padding and
ended sequences, every combination of norms, far positions, rows that are not stored, and that
nothing else of the cache or the outputs changes."""
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


from paged_common import EPS, HALF_BF16, THETA, Batch, turned  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402


def append(b, d, pos=None, norm_k=True, norm_q=True, with_q=True, in_place=False, theta=THETA):
    """The call on fresh copies of the cache; q_out is pre-filled."""
    k_pages, v_pages = d["k_pages"].clone(), d["v_pages"].clone()
    q = d["q"].clone()
    q_out = q if in_place else torch.full_like(q, 7.0)
    msa.msa_paged_append(d["k_new"], d["v_new"], q if with_q else None, d["q_off"], d["kv_len"], d["page_table"],
                         k_pages, v_pages, q_out if with_q else None, EPS, theta,
                         pos_off=None if pos is None else b.i32(pos), w_k=d["w_k"] if norm_k else None,
                         w_q=d["w_q"] if norm_q else None)
    torch.cuda.synchronize()
    return k_pages.cpu(), v_pages.cpu(), q_out.cpu()


def near(got, x, w, positions, theta=THETA):
    """One rounding to bf16 of values whose fp32 errors are at most 32 roundings of the two products
    behind each (norm factor, sine and cosine at 2^-23 each, their products and the sum)."""
    ref, size = turned(x, w, positions, theta=theta)
    err = (got.double() - ref).abs()
    tol = HALF_BF16 * ref.abs() + 1.01 * 32 * 2.0 ** -24 * size
    assert (err <= tol).all(), (err - tol).max()


def check(b, got, pos=None, norm_k=True, norm_q=True, with_q=True, dropped=(), theta=THETA, q_before=7.0):
    k_pages, v_pages, q_out = got
    pos = pos or [0] * b.B
    k_left, v_left = torch.ones(b.k_pages.shape[:3], dtype=torch.bool), torch.ones(b.k_pages.shape[:3], dtype=torch.bool)
    for s in range(b.B):
        n = b.new[s]
        if n == 0:
            continue
        mine = slice(b.q_off[s], b.q_off[s + 1])
        p = [pos[s] + b.rows[s] - n + i for i in range(n)]
        for l in range(b.L):
            kept = [i for i in range(n) if (s, i) not in dropped]
            if kept:
                spots = [b.spot(s, b.rows[s] - n + i) for i in kept]
                pg, rw = torch.tensor([x[0] for x in spots]), torch.tensor([x[1] for x in spots])
                at = torch.tensor(kept) + b.q_off[s]
                near(k_pages[l, pg, rw], b.k_new[l, at], b.w_k[l] if norm_k else None, [p[i] for i in kept], theta)
                assert torch.equal(v_pages[l, pg, rw], b.v_new[l, at])
                k_left[l, pg, rw] = v_left[l, pg, rw] = False
            if with_q:
                near(q_out[l, mine], b.q[l, mine], b.w_q[l] if norm_q else None, p, theta)
    # every other row of the cache and the padding rows of q_out are as they were
    assert torch.equal(k_pages.view(torch.int16)[k_left], b.k_pages.view(torch.int16)[k_left])
    assert torch.equal(v_pages.view(torch.int16)[v_left], b.v_pages.view(torch.int16)[v_left])
    if with_q:
        tail = q_out[:, b.q_off[-1]:]
        want = b.q[:, b.q_off[-1]:] if q_before is None else torch.full_like(tail, q_before)
        assert torch.equal(tail, want)


@pytest.mark.parametrize("new,rows,page,hq,layers,pad", [
    ([1], [1], 1, 8, 1, 0),
    ([1], [65], 64, 32, 18, 0),
    ([3, 0, 1, 17, 0], [3, 5, 90, 40, 0], 16, 32, 2, 3),
    ([0, 0, 130], [7, 0, 131], 32, 64, 1, 1),
    ([5, 64, 1, 33], [69, 64, 700, 50], 256, 16, 3, 0),
    ([2] * 70, list(range(2, 72)), 2, 8, 1, 5),
])
def test_append_ragged(new, rows, page, hq, layers, pad):
    print("case: append", new[:5], rows[:5], page, hq, layers, pad, flush=True)
    b = Batch(new, rows, page=page, hq=hq, layers=layers, pad=pad, seed=hash((page, hq, layers)) & 0xFFFF)
    d = b.to_device()
    pos = [(37 * s) % 101 for s in range(b.B)]
    check(b, append(b, d, pos), pos)


@pytest.mark.parametrize("norm_k,norm_q,with_q,in_place", [(False, False, True, False), (True, False, True, True),
                                                           (False, True, True, True), (True, False, False, False),
                                                           (False, False, False, False)])
def test_append_variants(norm_k, norm_q, with_q, in_place):
    print("case: append variants", norm_k, norm_q, with_q, in_place, flush=True)
    b = Batch([4, 1, 9], [20, 1, 33], page=8, hq=32, layers=2, pad=2, seed=5)
    got = append(b, b.to_device(), None, norm_k, norm_q, with_q, in_place)
    check(b, got, None, norm_k, norm_q, with_q, q_before=None if in_place else 7.0)


@pytest.mark.parametrize("theta", [1.0, 1e4, 1e6, 1e-2])
def test_append_far_positions(theta):
    """Angles of positions up to 2^31 keep their fraction of a turn (and negative ones, and theta <= 1)."""
    print("case: append far positions", theta, flush=True)
    b = Batch([3, 2, 2, 1], [9, 70, 5, 1], page=16, hq=8, seed=11)
    pos = [2 ** 31 - 20, 1 << 20, -300, -1]
    # the reference's angle p * theta^(-e/64) is itself off by p * theta^(-e/64) * 2^-52 or so: only
    # angles below 2^27 are compared (2^-25 then); theta 1e-2 stays below with the smaller positions
    if theta < 1:
        pos = [1 << 19, 1 << 16, -300, -1]
    else:
        pos[0] = (1 << 27) - 20
    check(b, append(b, b.to_device(), pos, theta=theta), pos, theta=theta)


def test_append_many_sequences():
    """More than 64 sequences (a second search step), most of them without a token."""
    print("case: append 2048 sequences", flush=True)
    rng = np.random.default_rng(3)
    new = rng.choice([0, 0, 0, 1, 2], 2048).tolist()
    rows = [n + int(rng.integers(0, 5)) for n in new]
    b = Batch(new, rows, page=4, hq=8, seed=9, pad=1)
    check(b, append(b, b.to_device()))


def test_append_rows_that_are_not_stored():
    """Rows below 0, past the page table's row and on pages outside the pool: nothing is written for
    them, the others are stored, and every query is turned."""
    print("case: append dropped rows", flush=True)
    b = Batch([4, 3, 2, 2], [10, 3, 18, 20], page=8, hq=16, seed=21)
    d = b.to_device()
    kv = [2, 3, 8 * b.max_pages + 1, 20]          # 2 rows of 4 tokens below 0; the last row past the table
    d["kv_len"] = b.i32(kv)
    d["page_table"] = d["page_table"].clone()
    d["page_table"][1, 0] = b.n_pages             # sequence 1: a page behind the pool
    d["page_table"][3, 2] = -5                    # sequence 3: rows 16 .. 23
    got = append(b, d)
    b.rows = kv
    b.table[2, b.max_pages - 1] = int(d["page_table"][2, b.max_pages - 1])
    check(b, got, dropped={(0, 0), (0, 1), (1, 0), (1, 1), (1, 2), (2, 1), (3, 0), (3, 1)})


def test_append_special_values():
    """Zeros stay zeros with a norm (eps keeps the factor finite), infinities and NaN stay in their head."""
    print("case: append special values", flush=True)
    b = Batch([3], [3], page=4, hq=8, seed=2)
    b.k_new[0, 0] = 0
    b.k_new[0, 1, 3, 5] = float("inf")
    b.k_new[0, 2, 6, 100] = float("nan")
    d = b.to_device()
    k_pages, v_pages, _ = append(b, d)
    rows = b.local(k_pages, 0, 0, 3)
    assert (rows[0] == 0).all()
    keep = torch.ones(8, dtype=torch.bool)
    keep[3] = False
    near(rows[1:2][:, keep], b.k_new[0, 1:2][:, keep], b.w_k[0], [1])
    keep[3], keep[6] = True, False
    near(rows[2:3][:, keep], b.k_new[0, 2:3][:, keep], b.w_k[0], [2])
    assert torch.isnan(rows[2, 6]).all()


def test_append_pool_beyond_32_bit_offsets():
    """The last pages of a pool of more than 2^32 bytes and 2^31 elements, on a second layer."""
    print("case: append into a 6.4 GB pool", flush=True)
    b = Batch([2, 3], [40, 3], page=64, hq=8, layers=2, seed=4)
    d = b.to_device()
    n_pages = 25000
    shift = n_pages - b.n_pages
    big = [torch.zeros(2, n_pages, 64, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    msa.msa_paged_append(d["k_new"], d["v_new"], None, d["q_off"], d["kv_len"], d["page_table"] + shift, big[0],
                         big[1], None, EPS, THETA, w_k=d["w_k"])
    torch.cuda.synchronize()
    for l in range(2):
        for s in range(2):
            for i in range(b.new[s]):
                pg, rw = b.spot(s, b.rows[s] - b.new[s] + i)
                at = b.q_off[s] + i
                near(big[0][l, pg + shift, rw].cpu()[None], b.k_new[l, at][None], b.w_k[l], [b.rows[s] - b.new[s] + i])
                assert torch.equal(big[1][l, pg + shift, rw].cpu(), b.v_new[l, at])
    assert int((big[1] != 0).any(-1).any(-1).sum()) == 2 * 5


def test_append_no_tokens():
    b = Batch([0, 0], [3, 4], page=4, hq=8, seed=1)
    d = b.to_device()
    check(b, append(b, d))
