"""GPU tests of the paged calls on some of a packed batch's sequences: q_off begins above 0 and ends before the last
row, and the rows of the other sequences are left as they were."""
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


from paged_common import EPS, THETA, Batch  # noqa: E402
from paged_exact import SCALE, check_every_token  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
BATCHES = [  # new, rows: cut into parts, so that a token's parts are described in the workspace
    ([1] * 8, [2000 + 50 * s for s in range(8)]),
    ([40, 1, 300, 1, 2, 0, 70, 1], [900, 800, 1000, 3000, 700, 30, 900, 1200]),
]


def call(d, out, ws, first=0, last=None):
    """Sequences first .. last) of the batch, in the packed arrays of all."""
    part = slice(first, last)
    off = d["q_off"][first:None if last is None else last + 1].contiguous()
    msa.msa_paged_attend(d["q"], off, d["kv_len"][part].contiguous(), d["page_table"][part].contiguous(), d["k_pages"],
                         d["v_pages"], SCALE, out, ws, ctx_k=d["ctx_k"][:, part].contiguous(),
                         ctx_v=d["ctx_v"][:, part].contiguous(), ctx_len=d["ctx_len"][:, part].contiguous())
    torch.cuda.synchronize()
    return off.cpu().tolist()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first,last", [(4, None), (2, 7), (7, 8), (3, 6)])
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_attend_some_sequences(case, first, last, dtype):
    """Right behind a call with all of them, in the workspace that it leaves."""
    print("case: some sequences", case, first, last, dtype, flush=True)
    new, rows = BATCHES[case]
    B = len(new)
    ctx = [[100 + 9 * s for s in range(B)]]
    b = Batch(new, rows, ctx=ctx, page=32, hq=32, pad=3, seed=600 + case)
    d = b.to_device()
    last = last or B
    ws = torch.empty(max(msa.msa_paged_attend_workspace_size(1, n, n, b.n_q, 32) for n in (B, last - first)),
                     dtype=torch.uint8, device="cuda")
    out = torch.full((1, b.n_q, 32, 128), 7.0, dtype=dtype, device="cuda")
    call(d, out, ws)
    out.fill_(7.0)
    off = call(d, out, ws, first, last)
    assert off[0] > 0
    assert (out[:, :off[0]] == 7.0).all(), "rows of the sequences before"
    assert (out[:, off[-1]:] == 7.0).all(), "rows of the sequences behind"
    part = slice(first, last)
    check_every_token(out, d["q"], off, rows[part], d["page_table"][part], d["k_pages"], d["v_pages"],
                      (d["ctx_k"][:, part], d["ctx_v"][:, part], [ctx[0][part]], list(range(last - first))))


def test_append_some_sequences():
    print("case: append some sequences", flush=True)
    new, rows = BATCHES[1]
    b = Batch(new, rows, page=32, hq=32, pad=3, seed=610)
    d = b.to_device()

    def append(part):
        k, v, q = d["k_pages"].clone(), d["v_pages"].clone(), torch.full_like(d["q"], 7.0)
        off = d["q_off"][part.start:part.stop + 1].contiguous()
        msa.msa_paged_append(d["k_new"], d["v_new"], d["q"], off, d["kv_len"][part].contiguous(),
                             d["page_table"][part].contiguous(), k, v, q, EPS, THETA, w_k=d["w_k"], w_q=d["w_q"])
        torch.cuda.synchronize()
        return k, v, q

    whole, some = append(slice(0, 8)), append(slice(2, 7))
    lo, hi = b.q_off[2], b.q_off[7]
    assert torch.equal(some[2][:, lo:hi], whole[2][:, lo:hi])
    assert (some[2][:, :lo] == 7.0).all() and (some[2][:, hi:] == 7.0).all()
    mine = torch.zeros(b.n_pages, b.page, dtype=torch.bool)
    for s in range(2, 7):
        for i in range(new[s]):
            mine[b.spot(s, rows[s] - new[s] + i)] = True
    mine = mine.cuda()
    for x, y, before in zip(some[:2], whole[:2], (d["k_pages"], d["v_pages"])):
        assert torch.equal(x[:, mine], y[:, mine]) and torch.equal(x[:, ~mine], before[:, ~mine])
