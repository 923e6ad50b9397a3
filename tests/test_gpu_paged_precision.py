"""GPU tests of what the paged calls' precision is: the weights of fp32 output in three bf16 parts, and a serving
loop whose every value is compared with 64 bits of what the calls themselves were given."""
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


from paged_common import HALF_BF16, turned  # noqa: E402
from paged_exact import check_every_token  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402
from test_gpu_paged_path import Server  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def bf16_parts(p, n):
    """What n bf16 values, each the rounding of what those before it leave, hold of p."""
    held = torch.zeros_like(p)
    for _ in range(n):
        held = held + (p - held).to(BF16).double()
    return held


@pytest.mark.parametrize("sequences,tokens,hq", [
    (1, 1, 64), (64, 1, 8), (23, 1, 32), (5, 3, 32),                          # streamed: up to 16 columns
    (1, 17, 8), (1, 30, 8), (3, 60, 8), (1, 16, 32), (2, 100, 8), (1, 70, 64)])   # shared tiles: 1, 2 and 4 blocks
def test_weights_keep_24_bits(sequences, tokens, hq):
    """Two rows: a score of 0 with V = 0, and a score of -j / 32 (j a whole number, the scale 1 / 32: both exact)
    with V = v.  The output is p v / (1 + p), p = exp(-j / 32).

    In units of 2^-24: log2 e (1/4) and its product with the score (1) are off by 5/4 of an exponent of up to 2.9
    (in the weight times ln 2: 2.6), exp2 by one step (2), three bf16 parts by 1/2: the weight by 5.1, the output by
    5.1 / (1 + p).  Its sum takes two additions next to an exact product (one step, 2, each), 1 + p one
    rounding, the division and the product with it one each: 7.  Two parts hold p but for up to 2^-17, 128 units,
    which the same bound refuses."""
    print("case: weights", sequences, tokens, hq, flush=True)
    n, G = sequences * tokens, hq // 8
    gen = torch.Generator().manual_seed(n + hq)
    j = 1 + (torch.arange(n * hq) * 37 + 5) % 64
    q = torch.zeros(1, n, hq, 128)
    q[0, :, :, 3] = -j.view(n, hq).float()
    ctx_k = torch.zeros(1, sequences, 2, 8, 128)
    ctx_k[:, :, 1, :, 3] = 1.0
    ctx_v = torch.zeros(1, sequences, 2, 8, 128)
    ctx_v[:, :, 1] = torch.rand(sequences, 8, 128, generator=gen) + 1.0
    ctx_v[:, :, 1] *= torch.randint(0, 2, ctx_v[:, :, 1].shape, generator=gen) * 2 - 1
    q, ctx_k, ctx_v = (t.to(BF16) for t in (q, ctx_k, ctx_v))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out = torch.empty(1, n, hq, 128, device="cuda")
    ws = torch.empty(msa.msa_paged_attend_workspace_size(1, sequences, sequences, n, hq), dtype=torch.uint8, device="cuda")
    pages = torch.zeros(1, 1, 16, 8, 128, dtype=BF16, device="cuda")
    msa.msa_paged_attend(q.cuda(), i32([tokens * s for s in range(sequences + 1)]), i32([0] * sequences),
                         i32([[0]] * sequences), pages, pages, 1 / 32, out, ws, ctx_k=ctx_k.cuda(), ctx_v=ctx_v.cuda(),
                         ctx_len=i32([[2] * sequences]))
    torch.cuda.synchronize()
    p = torch.exp(-j.double() / 32).view(n, hq, 1)
    v = ctx_v[0, :, 1].double().repeat_interleave(G, 1).repeat_interleave(tokens, 0)
    ref = p * v / (1 + p)
    tol = (5.1 / (1 + p) + 7) * U * ref.abs()
    over = ((out[0].cpu().double() - ref).abs() - tol).amax()
    assert over <= 0, "%g over its bound" % over
    two = bf16_parts(p.float().double(), 2) * v / (1 + p)
    assert ((two - ref).abs() > tol).any()


def test_serving_loop_to_the_last_value():
    """Prompts, then tokens, some sequences pausing: the rows and queries that each append writes, and the
    attention over just these rows."""
    print("case: serving loop, every value", flush=True)
    sv = Server(21)
    group = [0, 0, 0, 1, 1]
    ctx = (sv.ctx_k, sv.ctx_v, sv.ctx_len.tolist(), group)
    for new in ([20, 1, 7, 33, 0], [1, 1, 1, 1, 40], [1, 0, 1, 1, 1], [3, 1, 1, 0, 1], [1, 1, 1, 1, 1], [0, 60, 1, 2, 0]):
        x = sv.inputs(new)
        before = sv.k_pages.clone(), sv.v_pages.clone()
        sv.step(x)
        torch.cuda.synchronize()
        off, rows = x["q_off"].tolist(), sv.kv_len.tolist()
        old = torch.ones(sv.n_pages, sv.P, dtype=torch.bool, device="cuda")
        for s, n in enumerate(new):
            r = torch.arange(rows[s] - n, rows[s], device="cuda")
            page, row = sv.table[s].long()[r // sv.P], r % sv.P
            old[page, row] = False
            mine = slice(off[s], off[s + 1])
            assert torch.equal(sv.v_pages[:, page, row], x["v"][:, mine])
            for l in range(sv.L):
                for got, raw, w in ((sv.k_pages[l, page, row], x["k"][l, mine], sv.w_k[l]),
                                    (x["q_out"][l, mine], x["q"][l, mine], sv.w_q[l])):
                    ref, size = turned(raw.cpu(), w.cpu(), (r.cpu() + 16).tolist())
                    # one rounding to bf16 of values that are off by at most 32 fp32 roundings of their two products
                    tol = HALF_BF16 * ref.abs() + 1.01 * 32 * U * size
                    assert ((got.cpu().double() - ref).abs() <= tol).all(), (l, s)
        assert torch.equal(sv.k_pages[:, old], before[0][:, old]) and torch.equal(sv.v_pages[:, old], before[1][:, old])
        check_every_token(x["out"], x["q_out"], off, rows, sv.table, sv.k_pages, sv.v_pages, ctx)
