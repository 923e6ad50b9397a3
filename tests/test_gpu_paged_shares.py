"""GPU tests of how msa_paged_attend shares out the rows of many short sequences in many layers: a workgroup
lists 32 pieces of streams at a time, so shares of 31, 32, 33, 64 and 65 pieces, ending with a stream or inside
one.  Every token of every layer is compared with 64 bits."""
import random

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


from paged_exact import SCALE, check_every_token  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
PAGE = 32


def shares(jobs, layers):
    """Of each share of a layer's streams (two for each job of so many 32-row tiles; the shares of up to 512
    workgroups over the layers): how many pieces it holds, and whether its last stream goes on in the next."""
    ends, total = [], 0
    for t in jobs:
        for _ in range(2):
            total += t
            ends.append(total)
    wgs = max(1, 512 // layers)
    size = -(-total // wgs)
    out, first = [], 0
    for to in range(size, total + size, size):
        to = min(to, total)
        last = first
        while ends[last] < to:
            last += 1
        out.append((last - first + 1, ends[last] > to))
        first = last + (ends[last] == to)
    return out


def tiles(rows):
    return max(1, -(-rows // 32))


def batch(rows, layers, hq, seed, dtype, groups=None, lens=None, new=None):
    """One new token a sequence, or `new`; the sequences' pages are any of a small pool's."""
    B, most = len(rows), max(rows)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pool, q_off = 61, [0]
    for n in new or [1] * B:
        q_off.append(q_off[-1] + n)
    n_q = q_off[-1]
    q, k_pages, v_pages = normal(layers, n_q, hq, 128) * 2, *(normal(layers, pool, PAGE, 8, 128) for _ in range(2))
    table = torch.randint(0, pool, (B, -(-most // PAGE)), generator=gen, device="cuda", dtype=torch.int32)
    ctx, extra, n_groups = None, {}, B
    if groups:
        n_groups = len(groups)
        most_ctx = max(max(x) for x in lens)
        off = [0]
        for n in groups:
            off.append(off[-1] + n)
        ctx = (normal(layers, n_groups, most_ctx, 8, 128), normal(layers, n_groups, most_ctx, 8, 128), lens,
               [g for g, n in enumerate(groups) for _ in range(n)])
        extra = dict(grp_off=i32(off), ctx_k=ctx[0], ctx_v=ctx[1], ctx_len=i32(lens))
    out = torch.full((layers, n_q, hq, 128), 7.0, dtype=dtype, device="cuda")
    ws = torch.empty(msa.msa_paged_attend_workspace_size(layers, B, n_groups, n_q, hq), dtype=torch.uint8, device="cuda")
    msa.msa_paged_attend(q, i32(q_off), i32(rows), table, k_pages, v_pages, SCALE, out, ws.fill_(0xFF), **extra)
    torch.cuda.synchronize()
    check_every_token(out, q, q_off, rows, table, k_pages, v_pages, ctx)


@pytest.mark.parametrize("sequences,pieces,cut", [
    (422, 31, True), (421, 31, False), (437, 32, True), (443, 32, True), (447, 32, False), (451, 33, True), (885, 64, True),
    (899, 65, True)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shares_of_so_many_pieces(sequences, pieces, cut, dtype):
    print("case: shares of %d pieces" % pieces, sequences, cut, dtype, flush=True)
    rng = random.Random(sequences)
    rows = [rng.randint(65, 96) for _ in range(sequences)]
    assert (pieces, cut) in shares([3] * sequences, 18)
    batch(rows, 18, 32, sequences, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ragged_lengths(dtype):
    print("case: ragged lengths", dtype, flush=True)
    rng = random.Random(2)
    rows = [rng.randint(40, 400) for _ in range(220)]
    assert any(n % 32 == 0 and cut for n, cut in shares([tiles(r) for r in rows], 36))
    batch(rows, 36, 32, 1, dtype)


def test_groups():
    """Streams of the sequences' own rows, then those of the memory rows that each seven share."""
    print("case: shares in groups", flush=True)
    rng = random.Random(0)
    rows = [rng.randint(1, 90) for _ in range(7 * 40)]
    lens = [[rng.randint(1, 90) for _ in range(40)] for _ in range(24)]
    lists = [shares([tiles(r) for r in rows + c], 24) for c in lens]
    assert sum(any(n % 32 == 0 and cut for n, cut in x) for x in lists) >= 2
    batch(rows, 24, 8, 2, F32, groups=[7] * 40, lens=lens)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layers,sequences,grouped", [(18, 330, False), (18, 330, True), (36, 203, True), (8, 700, False)])
def test_streams_next_to_items(layers, sequences, grouped, dtype):
    """One token each, and one sequence in fifty brings more: shares of many pieces beside shared tiles."""
    print("case: streams next to items", layers, sequences, grouped, dtype, flush=True)
    rng = random.Random(sequences + layers)
    new = [rng.choice([17, 60, 140]) if s % 50 == 20 else 1 for s in range(sequences)]
    rows = [n + rng.randint(0, 130) for n in new]
    groups = [rng.randint(1, 9) for _ in range(sequences)] if grouped else None
    if grouped:
        groups = groups[:next(i for i in range(sequences) if sum(groups[:i]) >= sequences - 9)]
        groups.append(sequences - sum(groups))
    lens = [[rng.randint(0, 70) for _ in groups] for _ in range(layers)] if grouped else None
    batch(rows, layers, 32, sequences, dtype, groups=groups, lens=lens, new=new)
