"""CPU-side checks of the paged entry points: refusals through the C ABI and through the binding."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def msa():
    from routed_kv_memory_amd import msa as m
    m.lib()
    return m


P, F = ctypes.c_void_p, ctypes.c_float
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
fake, odd = P(0x1000), P(0x1002)


def append(msa, **change):
    a = dict(n_layers=1, B=2, n_q=3, Hq=32, k_new=fake, v_new=fake, q=fake, q_off=fake, kv_len=fake, pos_off=None,
             page_table=fake, max_pages=4, page_tokens=16, n_pages=9, w_k=None, w_q=None, eps=F(1e-6), theta=F(1e6),
             k_pages=fake, v_pages=fake, q_out=fake, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return msa.lib().msa_paged_append(*a.values())


def attend(msa, **change):
    a = dict(n_layers=1, B=2, n_groups=2, n_q=3, Hq=32, q=fake, q_off=fake, grp_off=None, ctx_k=None, ctx_v=None,
             ctx_len=None, max_ctx=0, k_pages=fake, v_pages=fake, n_pages=9, page_tokens=16, page_table=fake,
             max_pages=4, kv_len=fake, pre_len=None, scale=F(0.1), out_bf16=0, out=fake, workspace=fake,
             workspace_bytes=1 << 40, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return msa.lib().msa_paged_attend(*a.values())


@pytest.mark.parametrize("status,change", [
    (NULL, dict(k_new=None)), (NULL, dict(v_new=None)), (NULL, dict(q_off=None)), (NULL, dict(kv_len=None)),
    (NULL, dict(page_table=None)), (NULL, dict(k_pages=None)), (NULL, dict(v_pages=None)), (NULL, dict(q_out=None)),
    (SHAPE, dict(k_new=odd)), (SHAPE, dict(q=odd)), (SHAPE, dict(w_k=odd)), (SHAPE, dict(w_q=odd)),
    (SHAPE, dict(v_pages=odd)), (SHAPE, dict(q_out=odd)),
    (SHAPE, dict(n_layers=0)), (SHAPE, dict(B=0)), (SHAPE, dict(n_q=-1)), (SHAPE, dict(max_pages=0)),
    (SHAPE, dict(n_pages=0)), (SHAPE, dict(page_tokens=0)), (SHAPE, dict(page_tokens=24)),
    (SHAPE, dict(page_tokens=2048)), (SHAPE, dict(Hq=12)), (SHAPE, dict(Hq=0)), (UNSUPPORTED, dict(Hq=24)),
    (UNSUPPORTED, dict(Hq=128)), (UNSUPPORTED, dict(n_layers=65536)), (UNSUPPORTED, dict(B=2049)),
    (UNSUPPORTED, dict(n_q=(1 << 22) + 1)), (UNSUPPORTED, dict(max_pages=(1 << 26) + 1)),
    (UNSUPPORTED, dict(n_pages=1 << 27)),
    (SHAPE, dict(eps=F(-1.0))), (SHAPE, dict(eps=F(float("nan")))), (SHAPE, dict(theta=F(0.0))),
    (SHAPE, dict(theta=F(float("inf")))),
])
def test_append_refuses(msa, status, change):
    assert append(msa, **change) == status
    assert msa.lib().msa_last_error().startswith(b"msa_paged_append")


@pytest.mark.parametrize("status,change", [
    (NULL, dict(q=None)), (NULL, dict(q_off=None)), (NULL, dict(page_table=None)), (NULL, dict(kv_len=None)),
    (NULL, dict(k_pages=None)), (NULL, dict(v_pages=None)), (NULL, dict(out=None)), (NULL, dict(workspace=None)),
    (NULL, dict(max_ctx=8)), (NULL, dict(max_ctx=8, ctx_k=fake, ctx_v=fake)), (NULL, dict(n_groups=1)),
    (SHAPE, dict(q=odd)), (SHAPE, dict(out=odd)), (SHAPE, dict(k_pages=odd)),
    (SHAPE, dict(max_ctx=8, ctx_k=odd, ctx_v=fake, ctx_len=fake)),
    (SHAPE, dict(n_layers=0)), (SHAPE, dict(B=0)), (SHAPE, dict(n_groups=0)), (SHAPE, dict(n_groups=3)),
    (SHAPE, dict(n_q=-1)), (SHAPE, dict(max_ctx=-1)), (SHAPE, dict(Hq=20)), (UNSUPPORTED, dict(Hq=40)),
    (SHAPE, dict(page_tokens=48)), (SHAPE, dict(n_pages=0)), (SHAPE, dict(max_pages=0)),
    (SHAPE, dict(scale=F(0.0))), (SHAPE, dict(scale=F(-0.1))), (SHAPE, dict(scale=F(float("nan")))),
    (SHAPE, dict(scale=F(float("inf")))), (SHAPE, dict(out_bf16=2)),
    (UNSUPPORTED, dict(B=2049, n_groups=1, grp_off=fake)), (UNSUPPORTED, dict(n_q=(1 << 22) + 1)),
    (WORKSPACE, dict(workspace_bytes=16)),
])
def test_attend_refuses(msa, status, change):
    assert attend(msa, **change) == status
    assert msa.lib().msa_last_error().startswith(b"msa_paged_attend")


def test_no_tokens_enqueue_nothing(msa):
    assert append(msa, n_q=0, k_new=None, v_new=None, q=None, q_out=None, Hq=0) == OK
    assert attend(msa, n_q=0, q=None, out=None) == OK


def test_workspace_size(msa):
    f = msa.msa_paged_attend_workspace_size
    assert f(1, 1, 1, 1, 32) > 0 and f(18, 64, 8, 64, 32) > 0
    assert f(1, 2048, 1, 1 << 22, 64) > 0
    for bad in ((0, 1, 1, 1, 32), (1, 0, 1, 1, 32), (1, 1, 2, 1, 32), (1, 1, 0, 1, 32), (1, 1, 1, -1, 32), (1, 1, 1, 1, 24),
                (1, 2049, 1, 1, 32), (1, 1, 1, (1 << 22) + 1, 32)):
        assert f(*bad) == 0, bad


def cpu_args():
    bf, i = torch.bfloat16, torch.int32
    return {"k_new": torch.zeros(1, 3, 8, 128, dtype=bf), "v_new": torch.zeros(1, 3, 8, 128, dtype=bf),
            "q": torch.zeros(1, 3, 32, 128, dtype=bf), "q_off": torch.zeros(3, dtype=i), "kv_len": torch.zeros(2, dtype=i),
            "page_table": torch.zeros(2, 4, dtype=i), "k_pages": torch.zeros(1, 9, 16, 8, 128, dtype=bf),
            "v_pages": torch.zeros(1, 9, 16, 8, 128, dtype=bf), "q_out": torch.zeros(1, 3, 32, 128, dtype=bf)}


@pytest.mark.parametrize("name,value,error", [
    ("k_new", torch.zeros(3, 8, 128), ValueError), ("k_new", None, TypeError),
    ("v_new", torch.zeros(1, 2, 8, 128), ValueError), ("q", torch.zeros(1, 2, 32, 128), ValueError),
    ("q_out", None, ValueError), ("q_out", torch.zeros(1, 3, 16, 128), ValueError),
    ("q_off", torch.zeros(2, dtype=torch.int32), ValueError), ("kv_len", torch.zeros(3, dtype=torch.int32), ValueError),
    ("page_table", torch.zeros(8, dtype=torch.int32), ValueError), ("v_pages", torch.zeros(1, 8, 16, 8, 128), ValueError),
    ("k_pages", torch.zeros(2, 9, 16, 8, 128), ValueError),
    ("k_new", torch.zeros(1, 3, 8, 128, dtype=torch.float32), TypeError),      # dtype
    ("k_new", torch.zeros(1, 3, 8, 128, dtype=torch.bfloat16), ValueError),    # not on a GPU
])
def test_append_binding_refuses(msa, name, value, error):
    a = cpu_args()
    a[name] = value
    with pytest.raises(error):
        msa.msa_paged_append(a["k_new"], a["v_new"], a["q"], a["q_off"], a["kv_len"], a["page_table"], a["k_pages"],
                             a["v_pages"], a["q_out"], 1e-6, 1e6)


@pytest.mark.parametrize("change,error", [
    (dict(out=torch.zeros(1, 3, 16, 128)), ValueError), (dict(out=None), TypeError),
    (dict(grp_off=torch.zeros(2, 2, dtype=torch.int32)), ValueError),
    (dict(ctx_k=torch.zeros(1, 2, 8, 128)), ValueError),
    (dict(ctx_k=torch.zeros(1, 2, 5, 8, 128), ctx_v=None, ctx_len=torch.zeros(1, 2, dtype=torch.int32)), ValueError),
    (dict(ctx_k=torch.zeros(1, 3, 5, 8, 128), ctx_v=torch.zeros(1, 3, 5, 8, 128),
          ctx_len=torch.zeros(1, 3, dtype=torch.int32)), ValueError),
    (dict(pre_len=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(), ValueError),                                                      # not on a GPU
])
def test_attend_binding_refuses(msa, change, error):
    a = cpu_args()
    out = change.pop("out", torch.zeros(1, 3, 32, 128))
    with pytest.raises(error):
        msa.msa_paged_attend(a["q"], a["q_off"], a["kv_len"], a["page_table"], a["k_pages"], a["v_pages"], 0.1, out,
                             torch.zeros(8, dtype=torch.uint8), **change)


def test_attend_refuses_a_scale_past_the_range_of_its_scores(msa):
    assert attend(msa, scale=F(2.4e38)) == SHAPE
    assert attend(msa, scale=F(3.4e38)) == SHAPE
