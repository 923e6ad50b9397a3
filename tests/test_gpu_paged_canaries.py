"""Sentinels around the pages, outputs and workspace of the paged calls: nothing outside a buffer changes,
and the values do not depend on what the workspace held."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD, SENTINEL = 65536, 0xA5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from routed_kv_memory_amd import msa
    msa.lib()
    yield
    torch.cuda.synchronize()


from paged_common import EPS, SCALE, THETA, Batch, check_attention  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


class Guarded:
    def __init__(self, like=None, shape=None, dtype=None, fill=None):
        shape, dtype = (like.shape, like.dtype) if like is not None else (shape, dtype)
        self.n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((GUARD + self.n + GUARD,), SENTINEL, dtype=torch.uint8, device="cuda")
        if fill is not None:
            self.raw[GUARD:GUARD + self.n] = fill
        self.t = self.raw[GUARD:GUARD + self.n].view(dtype).view(shape)
        if like is not None:
            self.t.copy_(like)

    def check(self, name):
        torch.cuda.synchronize()
        assert (self.raw[:GUARD] == SENTINEL).all() and (self.raw[GUARD + self.n:] == SENTINEL).all(), name


BATCHES = [
    dict(new=[1], rows=[70], ctx=[[130]], page=16, hq=32),
    dict(new=[1, 0, 1, 2], rows=[40, 3, 900, 200], groups=[4], ctx=[[77]], pre=[32], page=16, hq=8),
    dict(new=[1] * 9, rows=[65 + s for s in range(9)], groups=[9], ctx=[[130]], pre=[64], page=32, hq=64),
    dict(new=[200, 1, 0, 17], rows=[260, 90, 4, 17], ctx=[[33, 0, 5, 64]], page=32, hq=32),
    dict(new=[1, 130, 1, 1, 60, 1], rows=[130, 258, 129, 140, 188, 131], groups=[4, 2], ctx=[[200, 31]], pre=[128, 100],
         page=4, hq=32),
    dict(new=[1] * 400, rows=[1 + s % 50 for s in range(400)], groups=[8] * 50, ctx=[[s % 40 for s in range(50)]], page=16,
         hq=32, layers=6),                      # its plan is made in a launch of its own
]


@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_nothing_around_the_buffers_changes(case):
    print("case: canaries", case, flush=True)
    a = dict(BATCHES[case])
    L = a.get("layers", 1)
    a["ctx"] = a["ctx"] * L
    b = Batch(pad=case % 3, seed=300 + case, q_std=2.0, **a)
    d = b.to_device()
    k_pages, v_pages, q = Guarded(d["k_pages"]), Guarded(d["v_pages"]), Guarded(d["q"])
    msa.msa_paged_append(d["k_new"], d["v_new"], q.t, d["q_off"], d["kv_len"], d["page_table"], k_pages.t, v_pages.t,
                         q.t, EPS, THETA, w_k=d["w_k"])
    for x, name in ((k_pages, "k_pages"), (v_pages, "v_pages"), (q, "q_out")):
        x.check(name)
    b.k_pages, b.v_pages, b.q = k_pages.t.cpu(), v_pages.t.cpu(), q.t.cpu()
    size = msa.msa_paged_attend_workspace_size(b.L, b.B, b.G, b.n_q, b.hq)
    for dtype in (F32, BF16):
        outs = []
        for fill in (0, 1, 0xFF):
            ws = Guarded(shape=(size,), dtype=torch.uint8, fill=fill)
            out = Guarded(shape=(b.L, b.n_q, b.hq, 128), dtype=dtype, fill=0)
            msa.msa_paged_attend(q.t, d["q_off"], d["kv_len"], d["page_table"], k_pages.t, v_pages.t, SCALE, out.t, ws.t,
                                 grp_off=d["grp_off"], ctx_k=d["ctx_k"], ctx_v=d["ctx_v"], ctx_len=d["ctx_len"],
                                 pre_len=d["pre_len"])
            ws.check("workspace")
            out.check("out")
            outs.append(out.t.clone())
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        live = [s for s in range(b.B) if b.new[s]]
        check_attention(b, outs[0], tokens=[(l, s, b.new[s] - 1) for l in {0, b.L - 1} for s in live[:8] + live[-4:]])


def test_captured_call_follows_its_lengths():
    """A call whose plan is a launch of its own, captured once: each replay sees the lengths of its time."""
    print("case: captured, many sequences", flush=True)
    b = Batch([1] * 400, [60 + s % 5 for s in range(400)], groups=[8] * 50, ctx=[[40] * 50] * 6, page=16, hq=32, layers=6,
              seed=401)
    d = b.to_device()
    ws = torch.empty(msa.msa_paged_attend_workspace_size(b.L, b.B, b.G, b.n_q, b.hq), dtype=torch.uint8, device="cuda")
    out, eager = (torch.zeros(b.L, b.n_q, b.hq, 128, device="cuda") for _ in range(2))

    def call(to):
        msa.msa_paged_attend(d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], SCALE, to, ws,
                             grp_off=d["grp_off"], ctx_k=d["ctx_k"], ctx_v=d["ctx_v"], ctx_len=d["ctx_len"])

    call(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    gen = torch.Generator().manual_seed(401)
    for step in range(4):
        lens = torch.randint(1, 65, (400,), generator=gen, dtype=torch.int32)
        d["kv_len"].copy_(lens.cuda())
        d["ctx_len"].copy_(torch.randint(0, 41, (6, 50), generator=gen, dtype=torch.int32).cuda())
        ws.fill_(step)
        call(eager)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step
