"""GPU tests of forms of the paged attention that a serving loop meets: the smallest and largest pages, a group whose
first sequence has ended, and a captured call whose groups change between replays."""
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


from paged_common import Batch  # noqa: E402
from paged_exact import SCALE, check_every_token  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def workspace(b):
    return torch.empty(msa.msa_paged_attend_workspace_size(b.L, b.B, b.G, b.n_q, b.hq), dtype=torch.uint8, device="cuda")


def attend(d, out, ws, grp_off):
    msa.msa_paged_attend(d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], SCALE, out, ws,
                         grp_off=grp_off, ctx_k=d["ctx_k"], ctx_v=d["ctx_v"], ctx_len=d["ctx_len"], pre_len=d["pre_len"])


def check(b, d, out, group_of=None):
    check_every_token(out, d["q"], b.q_off, d["kv_len"].tolist(), d["page_table"], d["k_pages"], d["v_pages"],
                      None if b.ctx is None else (d["ctx_k"], d["ctx_v"], b.ctx, group_of or b.group_of))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 512, 1024])
def test_page_sizes(page, dtype):
    """Streams, shared tiles of each width and a prefix that ends inside a page."""
    print("case: page size", page, dtype, flush=True)
    b = Batch([1, 2, 1, 140, 1, 9, 20], [400, 1203, 380, 1500, 65, 70, 333], groups=[3, 2, 1, 1], pre=[333, 0, 0, 0],
              ctx=[[40, 33, 0, 7]], page=page, hq=32, seed=700 + page, q_std=2.0)
    d = b.to_device()
    out = torch.full((1, b.n_q, 32, 128), 7.0, dtype=dtype, device="cuda")
    attend(d, out, workspace(b), d["grp_off"])
    torch.cuda.synchronize()
    check(b, d, out)


@pytest.mark.parametrize("length", [64, 20, 0])
@pytest.mark.parametrize("tokens", [1, 30])
def test_first_sequence_of_a_group_has_ended(tokens, length):
    """Its table still lists the shared pages, whatever its own length is."""
    print("case: first of the group ended", tokens, length, flush=True)
    b = Batch([0, tokens, 1, 0, 1], [64, 64 + tokens, 100, 64, 90], groups=[5], pre=[64], ctx=[[33]], page=16, hq=32,
              seed=710)
    d = b.to_device()
    d["kv_len"][0] = length
    for dtype in (F32, BF16):
        out = torch.full((1, b.n_q, 32, 128), 7.0, dtype=dtype, device="cuda")
        attend(d, out, workspace(b), d["grp_off"])
        torch.cuda.synchronize()
        check(b, d, out)


def test_captured_call_follows_its_groups():
    """Group slots as many as sequences: replays with a group for each, with one for all, with some idle."""
    print("case: captured, groups change", flush=True)
    b = Batch([1, 1, 20, 1, 140, 1], [300, 90, 64, 700, 150, 33], groups=[2, 0, 4, 0, 0, 0], ctx=[[100, 7, 300, 9, 0, 64]] * 3,
              page=16, hq=32, layers=3, seed=720)
    d = b.to_device()
    ws, out = workspace(b), torch.zeros(3, b.n_q, 32, 128, device="cuda")
    grp = b.i32(b.grp_off)
    attend(d, out, ws, grp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(d, out, ws, grp)
    for sizes in ([2, 0, 4, 0, 0, 0], [1] * 6, [6, 0, 0, 0, 0, 0], [0, 0, 0, 1, 2, 3], [1] * 6):
        off = [0]
        for n in sizes:
            off.append(off[-1] + n)
        grp.copy_(b.i32(off))
        ws.fill_(0x5A)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(b, d, out, [g for g, n in enumerate(sizes) for _ in range(n)])
