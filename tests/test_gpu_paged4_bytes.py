"""GPU tests of the paged local cache in 4 bits over all 256 scale bytes, those that the append does not write among
them: every code of every byte read back, and the attention over the smallest and the largest."""
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


import test_gpu_paged4_attend as attend_tests  # noqa: E402
from paged4_common import Batch4, pack, unpack, values  # noqa: E402
from routed_kv_memory_amd import msa  # noqa: E402

BF16 = torch.bfloat16


def test_read_every_code_of_every_scale_byte():
    """16 codes x 256 bytes, each where the low and where the high half of a byte is read; values past bf16's range are
    infinities."""
    print("case: read4, all scale bytes", flush=True)
    b = Batch4([64], [64], page=16, layers=1, seed=18)
    at = torch.arange(64 * 8 * 4).view(64, 8, 4)
    byte = (at % 256).to(torch.uint8)
    dim = torch.arange(32)
    code = ((dim + (at // 256)[..., None]) % 16).to(torch.uint8)      # each code in dims of either parity
    assert len({(int(s), int(c), int(p)) for s, cs in zip(byte.flatten(), code.flatten(0, 2))
                for c, p in zip(cs, dim % 2)}) == 256 * 16 * 2
    want = values(code.flatten(-2), byte).to(BF16)
    pages = b.k_pages4.clone()
    codes, scales = (t.clone() for t in unpack(pages))
    for r in range(64):
        page, row = b.spot(0, r)
        codes[0, page, row], scales[0, page, row] = code[r].flatten(-2), byte[r]
    d = b.to_device()
    pages = pack(codes, scales).cuda()
    k, v = (torch.empty(1, 64, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
    msa.msa_paged_read4(pages, pages, d["q_off"], d["page_table"], k, v)
    for got in (k[0].cpu(), v[0].cpu()):
        wrong = ~((got == want) | (got.isnan() & want.isnan())) | (torch.signbit(got) != torch.signbit(want)) & ~want.isnan()
        bad = wrong.view(64, 8, 4, 32)
        print("bytes with wrong values:", sorted({int(x) for x in byte[bad.any(-1)]}), flush=True)
        assert not wrong.any()


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("new", [1, 2, 7, 40])
@pytest.mark.parametrize("byte", [0, 1, 2, 252, 253, 254])
def test_values_of_every_size_reach_the_output(byte, new, dtype):
    """All rows alike, so an output is a row's values: bf16's subnormal numbers, the largest ones, infinities.  Streams
    and shared tiles."""
    print("case: attend4, scale byte", byte, new, dtype, flush=True)
    b = Batch4([new], [new], page=16, hq=64, layers=1, seed=19)
    code = (torch.arange(128) % 16).to(torch.uint8).expand(8, 128)
    codes, scales = (t.clone() for t in unpack(b.v_pages4))
    codes[:], scales[:] = code, byte
    b.v_pages4 = pack(codes, scales)
    k_codes, k_scales = (t.clone() for t in unpack(b.k_pages4))
    k_codes[:] = 0
    b.k_pages4 = pack(k_codes, k_scales)
    out = attend_tests.attend(b, dtype=dtype).cpu().double()[0]
    row = values(code, torch.full((8, 4), byte, dtype=torch.uint8)).to(BF16).double().repeat_interleave(8, 0)
    for t in range(new):
        want = row
        n = t + 1
        if byte >= 252 and n > 1:                 # sums past fp32's range are infinite
            continue
        # n equal weights: the sum, 1 / n and the product are rounded, each also to fp32's subnormal numbers
        bound = want.abs() * 4 * 2.0 ** -24 + 2.0 ** -149
        if dtype == BF16:
            bound = bound + (want.abs() + bound) * 2.0 ** -8 + 2.0 ** -134
        ok = torch.isfinite(want)
        assert torch.equal(out[t][~ok], want[~ok]), t
        assert bool(((out[t] - want).abs() <= bound)[ok].all()), (t, (out[t] - want).abs()[ok].max())


@pytest.mark.parametrize("new", [1, 2, 7, 40])
@pytest.mark.parametrize("byte", [0, 1, 2])
def test_small_keys_count(byte, new):
    """Keys that are bf16's subnormal numbers and queries near the largest: their scores decide the weights."""
    print("case: attend4, small keys, scale byte", byte, new, flush=True)
    b = Batch4([new], [70 + new], page=16, hq=64, layers=1, seed=20)
    codes, scales = (t.clone() for t in unpack(b.k_pages4))
    gen = torch.Generator().manual_seed(21 + byte)
    codes[:] = torch.randint(0, 16, codes.shape, generator=gen, dtype=torch.uint8)
    scales[:] = byte
    b.k_pages4, b.k_pages = pack(codes, scales), values(codes, scales).to(BF16)
    b.q = (b.q.float() * 2.0 ** (125 - byte)).to(BF16)
    attend_tests.check(b, attend_tests.attend(b))
