"""The append and the attention together, as a serving loop runs them: prompts, then one token at a
time over shared memory rows; the same step as a replayed graph; and calls on two streams at once."""
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


from paged_common import EPS, SCALE, THETA, Batch, attention, turned  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

BF16 = torch.bfloat16


class Server:
    """A cache of two layers for a batch of sequences in two groups; what was appended is kept on the
    host as the cache's own rounded rows."""

    def __init__(self, seed=3):
        self.L, self.B, self.P, self.hq, self.G = 2, 5, 16, 32, 2
        self.n_pages, self.max_pages = 80, 12
        gen = torch.Generator().manual_seed(seed)
        self.gen = gen
        r = lambda *s: torch.randn(*s, generator=gen).to(BF16).cuda()
        self.rand = r
        self.k_pages, self.v_pages = r(self.L, self.n_pages, self.P, 8, 128), r(self.L, self.n_pages, self.P, 8, 128)
        perm = torch.randperm(self.n_pages, generator=gen)[:self.B * self.max_pages].view(self.B, self.max_pages)
        self.table = perm.to(torch.int32).cuda()
        self.kv_len = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        self.pos = torch.full((self.B,), 16, dtype=torch.int32, device="cuda")
        self.grp = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
        self.ctx_k, self.ctx_v = r(self.L, self.G, 90, 8, 128), r(self.L, self.G, 90, 8, 128)
        self.ctx_len = torch.tensor([[70, 90], [13, 0]], dtype=torch.int32, device="cuda")
        self.w_k, self.w_q = r(self.L, 128), r(self.L, 128)

    def inputs(self, new):
        n = sum(new)
        off = [0]
        for x in new:
            off.append(off[-1] + x)
        return {"new": torch.tensor(new, dtype=torch.int32, device="cuda"),
                "q_off": torch.tensor(off, dtype=torch.int32, device="cuda"), "k": self.rand(self.L, n, 8, 128),
                "v": self.rand(self.L, n, 8, 128), "q": self.rand(self.L, n, self.hq, 128),
                "q_out": torch.empty(self.L, n, self.hq, 128, dtype=BF16, device="cuda"),
                "out": torch.empty(self.L, n, self.hq, 128, dtype=torch.float32, device="cuda"),
                "ws": torch.empty(msa.msa_paged_attend_workspace_size(self.L, self.B, self.G, n, self.hq),
                                  dtype=torch.uint8, device="cuda")}

    def step(self, x):
        self.kv_len += x["new"]
        msa.msa_paged_append(x["k"], x["v"], x["q"], x["q_off"], self.kv_len, self.table, self.k_pages, self.v_pages,
                             x["q_out"], EPS, THETA, pos_off=self.pos, w_k=self.w_k, w_q=self.w_q)
        msa.msa_paged_attend(x["q_out"], x["q_off"], self.kv_len, self.table, self.k_pages, self.v_pages, SCALE,
                             x["out"], x["ws"], grp_off=self.grp, ctx_k=self.ctx_k, ctx_v=self.ctx_v,
                             ctx_len=self.ctx_len)


def reference(sv, x, history):
    """Checks one step against 64 bits: `history` is each sequence's raw (k, v) rows so far, on the host."""
    new, off = x["new"].tolist(), x["q_off"].tolist()
    k, v, q = x["k"].cpu(), x["v"].cpu(), x["q"].cpu()
    out = x["out"].cpu()
    for s in range(sv.B):
        history[s][0].append(k[:, off[s]:off[s + 1]])
        history[s][1].append(v[:, off[s]:off[s + 1]])
    for l in range(sv.L):
        for s in range(sv.B):
            if not new[s]:
                continue
            hk, hv = (torch.cat(h, 1)[l] for h in history[s])
            rows = hk.shape[0]
            p = [16 + i for i in range(rows)]
            kk = turned(hk, sv.w_k[l].cpu(), p)[0].to(BF16)
            qq = turned(q[l, off[s]:off[s + 1]], sv.w_q[l].cpu(), p[rows - new[s]:])[0].to(BF16)
            b = Batch([new[s]], [rows], page=rows, hq=sv.hq, ctx=[[int(sv.ctx_len[l, 0 if s < 3 else 1])]], max_ctx=90)
            g = 0 if s < 3 else 1
            b.ctx_k, b.ctx_v = sv.ctx_k[l, g].cpu()[None, None], sv.ctx_v[l, g].cpu()[None, None]
            b.k_pages, b.v_pages, b.q = kk[None, None], hv[None, None], qq[None]
            b.table[:] = 0
            for i in range(new[s]):
                ref, tol = attention(b, 0, 0, i)
                # a value of the cache or the query next to a rounding border may have gone the other
                # way: one bf16 step (2^-7 relative) of a single factor moves a score by up to
                # 2^-7 max|q k| scale and the output by at most twice that; a handful of the 128 of a
                # row may (fp32 is off by 2^-20 of a value here: one value in some hundreds)
                qk = (qq[i].double().abs().amax() * kk.double().abs().amax()) * SCALE
                slack = 4 * 2 * 2.0 ** -7 * qk * hv.double().abs().amax()
                err = (out[l, off[s] + i].double() - ref).abs()
                assert (err <= tol + slack).all()
                # and most rows have no such flip
                assert (err <= tol).double().mean() > 0.5


def test_serving_loop():
    print("case: prompts, then tokens", flush=True)
    sv = Server()
    history = [([], []) for _ in range(sv.B)]
    for new in ([20, 1, 7, 33, 0], [1, 1, 1, 1, 40], [1, 0, 1, 1, 1], [3, 1, 1, 0, 1], [1, 1, 1, 1, 1]):
        x = sv.inputs(new)
        sv.step(x)
        torch.cuda.synchronize()
        reference(sv, x, history)


def test_captured_step_replays_like_the_eager_one():
    """kv_len is advanced inside the graph: each replay appends the next row and attends to it.  Eager work
    runs between the replays; every replay's outputs and cache equal the eager loop's, bit for bit."""
    print("case: captured step", flush=True)
    eager, graph = Server(7), Server(7)
    first = [30, 2, 9, 17, 1]
    a = eager.inputs(first)
    b = {k: v.clone() for k, v in a.items()}
    eager.step(a)
    graph.step(b)
    xe = eager.inputs([1, 1, 0, 1, 1])
    xg = {k: v.clone() for k, v in xe.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step(xg)
    for rep in range(4):
        eager.step(xe)
        want = [t.clone() for t in (xe["out"], xe["q_out"], eager.k_pages, eager.v_pages, eager.kv_len)]
        xe["ws"].fill_(0xA5)
        xg["ws"].fill_(0x5A)
        xg["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = (xg["out"], xg["q_out"], graph.k_pages, graph.v_pages, graph.kv_len)
        for u, w in zip(got, want):
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), rep
        for name in ("k", "v", "q"):              # the next token's inputs, at the same addresses
            xe[name].copy_(eager.rand(*xe[name].shape))
            xg[name].copy_(xe[name])


def test_two_streams_at_once():
    """Two steps of two servers, each on its own stream with its own workspace, give what they give alone."""
    print("case: two streams", flush=True)
    alone, both = [Server(11), Server(12)], [Server(11), Server(12)]
    xs = [s.inputs([60, 1, 2, 5, 40]) for s in alone]
    ys = [{k: v.clone() for k, v in x.items()} for x in xs]
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
        assert torch.equal(s.k_pages.view(torch.int16), t.k_pages.view(torch.int16))


def test_stream_argument():
    """The stream that is passed is the one that is used."""
    sv = Server(13)
    x = sv.inputs([1, 2, 3, 4, 5])
    want = {k: v.clone() for k, v in x.items()}
    sv.step(want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    msa.msa_paged_append(x["k"], x["v"], x["q"], x["q_off"], sv.kv_len, sv.table, sv.k_pages, sv.v_pages, x["q_out"], EPS,
                         THETA, pos_off=sv.pos, w_k=sv.w_k, w_q=sv.w_q, stream=st)
    msa.msa_paged_attend(x["q_out"], x["q_off"], sv.kv_len, sv.table, sv.k_pages, sv.v_pages, SCALE, x["out"], x["ws"],
                         grp_off=sv.grp, ctx_k=sv.ctx_k, ctx_v=sv.ctx_v, ctx_len=sv.ctx_len, stream=st)
    st.synchronize()
    assert torch.equal(x["out"], want["out"])


def test_captured_attends_with_one_workspace_in_sequence():
    """Two captured graphs that share a workspace, replayed one after the other on one stream."""
    print("case: two graphs, one workspace", flush=True)
    sv = Server(14)
    x, y = sv.inputs([9, 1, 1, 2, 1]), sv.inputs([1, 1, 30, 1, 1])
    big = max(x["ws"].numel(), y["ws"].numel())
    ws = torch.empty(big, dtype=torch.uint8, device="cuda")
    sv.kv_len += 50

    def run(z):
        msa.msa_paged_attend(z["q"], z["q_off"], sv.kv_len, sv.table, sv.k_pages, sv.v_pages, SCALE, z["out"], ws,
                             grp_off=sv.grp, ctx_k=sv.ctx_k, ctx_v=sv.ctx_v, ctx_len=sv.ctx_len)

    want = []
    for z in (x, y):
        run(z)
        torch.cuda.synchronize()
        want.append(z["out"].clone())
    graphs = []
    for z in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(z)
        graphs.append(g)
    for _ in range(3):
        for z in (x, y):
            z["out"].zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x["out"], want[0]) and torch.equal(y["out"], want[1])
