"""CPU-side checks of the entry points of the paged local cache held in 4 bits: the refusals through the C ABI
and through the binding, and the format's definition as the tests use it."""
import ctypes

import pytest
import torch

from paged4_common import pack, quantise, unpack, values

P, F = ctypes.c_void_p, ctypes.c_float
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
fake, odd = P(0x1000), P(0x1002)


@pytest.fixture(scope="module")
def msa():
    from routed_kv_memory_amd import msa as m
    m.lib()
    return m


def append(msa, **change):
    a = dict(n_layers=1, B=2, n_q=3, Hq=32, k_new=fake, v_new=fake, q=fake, q_off=fake, kv_len=fake, pos_off=None,
             page_table=fake, max_pages=4, page_tokens=16, n_pages=9, w_k=None, w_q=None, eps=F(1e-6), theta=F(1e6),
             k_pages=fake, v_pages=fake, q_out=fake, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return msa.lib().msa_paged_append4(*a.values())


def read(msa, **change):
    a = dict(n_layers=1, B=2, n_rows=3, row_off=fake, row0=None, page_table=fake, max_pages=4, page_tokens=16,
             n_pages=9, k_pages=fake, v_pages=fake, k_out=fake, v_out=fake, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return msa.lib().msa_paged_read4(*a.values())


def attend(msa, **change):
    a = dict(n_layers=1, B=2, n_groups=2, n_q=3, Hq=32, q=fake, q_off=fake, grp_off=None, ctx_k=None, ctx_v=None,
             ctx_len=None, max_ctx=0, k_pages=fake, v_pages=fake, n_pages=9, page_tokens=16, page_table=fake,
             max_pages=4, kv_len=fake, pre_len=None, scale=F(0.1), out_bf16=0, out=fake, workspace=fake,
             workspace_bytes=1 << 40, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return msa.lib().msa_paged_attend4(*a.values())


SIZES = [
    (SHAPE, dict(n_layers=0)), (SHAPE, dict(B=0)), (SHAPE, dict(max_pages=0)), (SHAPE, dict(n_pages=0)),
    (SHAPE, dict(page_tokens=0)), (SHAPE, dict(page_tokens=24)), (SHAPE, dict(page_tokens=2048)),
    (UNSUPPORTED, dict(n_layers=65536)), (UNSUPPORTED, dict(B=2049)),
    (UNSUPPORTED, dict(max_pages=(1 << 26) + 1)), (UNSUPPORTED, dict(n_pages=1 << 27)),
    (NULL, dict(page_table=None)), (NULL, dict(k_pages=None)), (NULL, dict(v_pages=None)),
    (SHAPE, dict(k_pages=odd)), (SHAPE, dict(v_pages=odd)),
]


@pytest.mark.parametrize("status,change", SIZES + [
    (NULL, dict(k_new=None)), (NULL, dict(v_new=None)), (NULL, dict(q_off=None)), (NULL, dict(kv_len=None)),
    (NULL, dict(q_out=None)), (SHAPE, dict(k_new=odd)), (SHAPE, dict(q=odd)), (SHAPE, dict(w_k=odd)),
    (SHAPE, dict(w_q=odd)), (SHAPE, dict(q_out=odd)), (SHAPE, dict(n_q=-1)), (SHAPE, dict(Hq=12)), (SHAPE, dict(Hq=0)),
    (UNSUPPORTED, dict(Hq=24)), (UNSUPPORTED, dict(Hq=128)), (UNSUPPORTED, dict(n_q=(1 << 22) + 1)),
    (SHAPE, dict(eps=F(-1.0))), (SHAPE, dict(eps=F(float("nan")))), (SHAPE, dict(theta=F(-1.0))),
    (SHAPE, dict(theta=F(float("nan")))), (SHAPE, dict(theta=F(float("inf")))),
])
def test_append_refuses(msa, status, change):
    assert append(msa, **change) == status
    assert msa.lib().msa_last_error().startswith(b"msa_paged_append4")


@pytest.mark.parametrize("status,change", SIZES + [
    (NULL, dict(row_off=None)), (NULL, dict(k_out=None)), (NULL, dict(v_out=None)), (SHAPE, dict(k_out=odd)),
    (SHAPE, dict(v_out=odd)), (SHAPE, dict(n_rows=-1)), (UNSUPPORTED, dict(n_rows=(1 << 22) + 1)),
])
def test_read_refuses(msa, status, change):
    assert read(msa, **change) == status
    assert msa.lib().msa_last_error().startswith(b"msa_paged_read4")


@pytest.mark.parametrize("status,change", [
    (st, ch) for st, ch in SIZES if "B" not in ch] + [
    (SHAPE, dict(B=0)), (UNSUPPORTED, dict(B=2049, n_groups=1, grp_off=fake)),
    (NULL, dict(q=None)), (NULL, dict(q_off=None)), (NULL, dict(kv_len=None)), (NULL, dict(out=None)),
    (NULL, dict(workspace=None)), (NULL, dict(max_ctx=8)), (NULL, dict(max_ctx=8, ctx_k=fake, ctx_v=fake)),
    (NULL, dict(n_groups=1)), (SHAPE, dict(q=odd)), (SHAPE, dict(out=odd)),
    (SHAPE, dict(max_ctx=8, ctx_k=odd, ctx_v=fake, ctx_len=fake)), (SHAPE, dict(n_groups=0)), (SHAPE, dict(n_groups=3)),
    (SHAPE, dict(n_q=-1)), (SHAPE, dict(max_ctx=-1)), (SHAPE, dict(Hq=20)), (UNSUPPORTED, dict(Hq=40)),
    (SHAPE, dict(scale=F(0.0))), (SHAPE, dict(scale=F(float("nan")))), (SHAPE, dict(scale=F(float("inf")))),
    (SHAPE, dict(out_bf16=2)), (UNSUPPORTED, dict(n_q=(1 << 22) + 1)), (WORKSPACE, dict(workspace_bytes=16)),
])
def test_attend_refuses(msa, status, change):
    assert attend(msa, **change) == status
    assert msa.lib().msa_last_error().startswith(b"msa_paged_attend4")


def test_attend_workspace(msa):
    size = msa.msa_paged_attend4_workspace_size
    assert size(18, 16, 1, 16, 32) > 0 and size(18, 16, 1, 16, 32) == msa.msa_paged_attend_workspace_size(18, 16, 1, 16, 32)
    assert size(1, 2, 3, 1, 32) == size(1, 0, 1, 1, 32) == size(1, 1, 1, 1, 24) == 0
    assert attend(msa, workspace_bytes=size(1, 2, 2, 3, 32) - 1) == WORKSPACE


def test_no_rows_enqueue_nothing(msa):
    assert append(msa, n_q=0, k_new=None, v_new=None, q=None, q_out=None) == OK
    assert append(msa, n_q=0, theta=F(0.0)) == OK
    assert read(msa, n_rows=0, k_out=None, v_out=None) == OK
    assert attend(msa, n_q=0, q=None, out=None) == OK


def test_the_binding_refuses(msa):
    """What the binding can see without a GPU: sizes that do not fit each other, wrong types, host tensors."""
    bf, i32 = torch.bfloat16, torch.int32
    rows, off, one = torch.zeros(1, 3, 8, 128, dtype=bf), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    table = torch.zeros(2, 4, dtype=i32)
    pages = torch.zeros(1, 9, 16 * 544, dtype=torch.uint8)
    good = [rows, rows, None, off, one, table, pages, pages, None, 1e-6, 1e6]
    for at, bad, error in ((6, pages[..., :-1].contiguous(), ValueError), (6, pages[0], ValueError), (6, None, TypeError),
                           (1, None, ValueError), (0, rows.float(), TypeError), (5, table[0], ValueError)):
        args = list(good)
        args[at] = bad
        with pytest.raises(error):
            msa.msa_paged_append4(*args)
    with pytest.raises(ValueError, match="GPU"):
        msa.msa_paged_append4(*good)
    good = [pages, pages, off, table, rows, rows]
    for at, bad, error in ((0, pages[..., :-1].contiguous(), ValueError), (2, one, ValueError), (2, off.long(), TypeError),
                           (4, rows[0], ValueError), (5, None, ValueError), (1, None, ValueError), (3, None, TypeError)):
        args = list(good)
        args[at] = bad
        with pytest.raises(error):
            msa.msa_paged_read4(*args)
    with pytest.raises(ValueError, match="GPU"):
        msa.msa_paged_read4(*good)


def test_row_bytes(msa):
    assert msa.ROW4_BYTES == 8 * (128 // 2 + 128 // 32) == 544


def test_the_format_of_the_tests():
    """Every value that a code stands for is held as itself, borders go to the even index, and pages are
    taken apart as they were put together.  A value is off by half the distance of its neighbours at most, 2^e between
    4 and 6 and from 6 to 7; e is the smallest, so the largest value m > 7 * 2^(e - 1): off by less than m / 3.5."""
    x = torch.zeros(8, 128, dtype=torch.float64)
    x[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x[1, :4] = torch.tensor([7.0, -7.0, 6.9, 0.5])
    x[2, :2] = torch.tensor([7.000001, 1.0])
    x[3, 40] = float("inf")
    x[4] = 1e-60
    x[5, 100] = -1e60
    codes, scales = quantise(x)
    assert codes[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7] and scales[0].tolist() == [127, 2, 2, 2]
    assert codes[1, :4].tolist() == [7, 15, 7, 1] and scales[1, 0] == 127
    assert codes[2, :2].tolist() == [6, 1] and scales[2, 0] == 128          # 3.5000005 -> 4, 0.5
    assert scales[3].tolist() == [2, 255, 2, 2]
    assert (codes[4] == 0).all() and (scales[4] == 2).all()
    assert codes[5, 100] == 15 and scales[5, 3] == 252
    g = torch.Generator().manual_seed(1)
    y = torch.randn(2, 3, 4, 8, 128, generator=g, dtype=torch.float64)
    codes, scales = quantise(y)
    held = values(codes, scales)
    assert torch.equal(held.to(torch.bfloat16).double(), held)
    again = quantise(held)
    assert torch.equal(values(*again), held)
    top = y.abs().unflatten(-1, (4, 32)).amax(-1)
    err = (held - y).abs().unflatten(-1, (4, 32)).amax(-1)
    assert (err < top / 3.5).all()
    pages = pack(codes, scales)
    assert pages.shape == (2, 3, 4 * 544)
    for a, b in zip(unpack(pages), (codes, scales)):
        assert torch.equal(a, b)
