"""GPU tests of groups given with as many slots as there are sequences (some then hold none): the group offsets
decide which memory rows a sequence sees, as they do with fewer slots."""
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
GUARD = 1 << 16


def attend(b, d, dtype, grp_off):
    """The call in a workspace of just its size; nothing behind it and no row behind the last sequence changes."""
    size = msa.msa_paged_attend_workspace_size(b.L, b.B, b.G, b.n_q, b.hq)
    ws = torch.full((size + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((b.L, b.n_q, b.hq, 128), 7.0, dtype=dtype, device="cuda")
    msa.msa_paged_attend(d["q"], d["q_off"], d["kv_len"], d["page_table"], d["k_pages"], d["v_pages"], SCALE, out,
                         ws[:size], grp_off=grp_off, ctx_k=d["ctx_k"], ctx_v=d["ctx_v"], ctx_len=d["ctx_len"],
                         pre_len=d["pre_len"])
    torch.cuda.synchronize()
    assert (ws[size:] == 0xFF).all() and (out[:, b.q_off[-1]:] == 7.0).all()
    return out[:, :b.q_off[-1]]


def check(b, d, out):
    check_every_token(out, d["q"][:, :b.q_off[-1]], b.q_off, b.rows, d["page_table"], d["k_pages"], d["v_pages"],
                      None if b.ctx is None else (d["ctx_k"], d["ctx_v"], b.ctx, b.group_of))


CASES = [  # new, rows, groups, pre, hq
    ([1, 1], [40, 70], [2, 0], None, 32),
    ([1, 1], [40, 70], [0, 2], [0, 32], 8),
    ([1, 2, 1], [33, 64, 100], [3, 0, 0], [32, 9, 0], 32),
    ([1, 1, 1], [33, 64, 100], [0, 0, 3], None, 64),
    ([1, 0, 1, 1], [40, 3, 1, 200], [0, 3, 1, 0], None, 16),
    ([5, 1, 20], [90, 64, 70], [2, 0, 1], [48, 64, 0], 32),
    ([1] * 9, [65 + s for s in range(9)], [9] + [0] * 8, [64] + [0] * 8, 32),
    ([1, 200, 1, 1, 130, 3], [90, 300, 91, 99, 230, 70], [4, 0, 0, 2, 0, 0], [64, 0, 0, 50, 0, 0], 32),
    ([128, 129, 1, 1], [200, 200, 200, 130], [0, 4, 0, 0], [0, 100, 0, 0], 32),
    ([600], [700], [1], [64], 64),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ctx", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_as_many_groups_as_sequences(case, ctx, dtype):
    print("case: groups", case, ctx, dtype, flush=True)
    new, rows, groups, pre, hq = CASES[case]
    assert len(groups) == len(new)
    lens = [[(37 * g + 61 * l + 11 * case) % 130 for g in range(len(groups))] for l in range(2)]
    b = Batch(new, rows, groups=groups, ctx=lens if ctx else None, pre=pre, page=16, hq=hq, layers=2, pad=case % 3,
              seed=500 + case, q_std=2.0)
    d = b.to_device()
    check(b, d, attend(b, d, dtype, b.i32(b.grp_off)))


def test_many_slots():
    """400 sequences in 50 of 400 slots, 6 layers: the plan is a launch of its own."""
    print("case: many slots", flush=True)
    groups = ([8] + [0] * 7) * 50
    b = Batch([1] * 400, [1 + s % 50 for s in range(400)], groups=groups,
              ctx=[[(s + l) % 40 for s in range(400)] for l in range(6)], page=16, hq=32, layers=6, seed=520)
    d = b.to_device()
    check(b, d, attend(b, d, F32, d["grp_off"]))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_each_sequence_its_own_group(dtype):
    """Given as offsets or not: the same bits."""
    print("case: own groups", dtype, flush=True)
    b = Batch([1, 300, 1, 40, 0, 2], [900, 333, 64, 40, 5, 600], ctx=[[70, 0, 333, 12, 9, 1000]], page=16, hq=32, seed=530)
    d = b.to_device()
    x, y = attend(b, d, dtype, None), attend(b, d, dtype, b.i32(b.grp_off))
    check(b, d, x)
    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("columns", [17, 32, 33, 64, 65, 96, 128, 129, 161, 193, 257])
def test_columns_of_a_shared_job(columns, dtype):
    """So many one-token sequences of one head per KV head, sharing rows that are cut into chunks: the parts of 32,
    64 and 128 columns side by side, in a workspace of just its size."""
    print("case: shared columns", columns, dtype, flush=True)
    other = [3, 1, 40]
    b = Batch([1] * columns + other, [300 + s % 7 for s in range(columns)] + [90, 30, 70], groups=[columns, 3],
              ctx=[[900, 33]], pre=[256, 0], page=64, hq=8, seed=540 + columns, q_std=2.0)
    d = b.to_device()
    check(b, d, attend(b, d, dtype, d["grp_off"]))
