"""Shared by the tests of the paged local cache held in 4 bits: the format in 64 bits, written from its
definition, and batches whose pages hold it."""
import torch

from paged_common import SCALE, Batch
from paged_exact import attend64

ROW4 = 544
ELEMENTS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def exponents(m):
    """The smallest e with m <= 7 * 2^e, in [-125, 125], by trying all of them."""
    e = torch.arange(-125, 126, dtype=torch.float64, device=m.device)
    return (-125 + (m[..., None] > 7 * torch.exp2(e)).sum(-1)).clamp(max=125)


def quantise(x):
    """Rows x [..., 128] in 64 bits: codes [..., 128] and scale bytes [..., 4]."""
    if x.numel() > 1 << 22 and x.dim() > 1:        # in pieces: the distances take 64 bytes a value
        parts = [quantise(p) for p in x.flatten(0, -2).split(1 << 15)]
        return tuple(torch.cat([p[i] for p in parts]).view(*x.shape[:-1], -1) for i in range(2))
    b = x.double().unflatten(-1, (4, 32))
    odd = ~torch.isfinite(b).all(-1)
    b = torch.where(odd[..., None], 0.0, b)
    e = exponents(b.abs().amax(-1))
    y = b.abs() * torch.exp2(-e.double())[..., None]
    d = (y[..., None] - ELEMENTS.to(x.device)).abs()
    near = d == d.amin(-1, keepdim=True)
    first = near.int().argmax(-1)
    code = first + ((first % 2 == 1) & (near.sum(-1) > 1))          # of two as near the even index
    code = torch.where(y > 6, 7, code) + 8 * torch.signbit(b).long()
    code = torch.where(odd[..., None], 0, code)
    return code.flatten(-2).to(torch.uint8), torch.where(odd, 255, e + 127).to(torch.uint8)


def values(codes, scales):
    """What codes [..., 128] and scale bytes [..., 4] stand for, in 64 bits."""
    codes = codes.long()
    x = ELEMENTS.to(codes.device)[codes & 7] * torch.where(codes >= 8, -1.0, 1.0).double()
    unit = torch.where(scales == 255, torch.nan, torch.exp2(scales.double() - 127))
    return (x.unflatten(-1, (4, 32)) * unit[..., None]).flatten(-2)


def pack(codes, scales):
    """Rows [L][n_pages][P][8][128] (and [4]) as pages [L][n_pages][544 P]."""
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return torch.cat([b.transpose(2, 3).flatten(2), scales.transpose(2, 3).flatten(2)], -1).contiguous()


def unpack(pages):
    """Pages [L][n_pages][544 P] as codes [L][n_pages][P][8][128] and scale bytes [..., 4]."""
    P = pages.shape[2] // ROW4
    b = pages[..., :512 * P].unflatten(-1, (8, P, 64)).transpose(2, 3)
    codes = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return codes, pages[..., 512 * P:].unflatten(-1, (8, P, 4)).transpose(2, 3)


class Batch4(Batch):
    """A Batch whose pages are held in 4 bits: k_pages4, v_pages4 are the bytes, k_pages, v_pages (bf16) the values
    they stand for."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        for name in ("k_pages", "v_pages"):
            self.hold(name, getattr(self, name))

    def hold(self, name, rows):
        codes, scales = quantise(rows.to(self.device))
        setattr(self, name + "4", pack(codes, scales).cpu())
        setattr(self, name, values(codes, scales).to(torch.bfloat16).cpu())

    def to_device(self):
        d = super().to_device()
        d["k_pages"], d["v_pages"] = self.k_pages4.to(self.device), self.v_pages4.to(self.device)
        return d


def check_every_token(out, q, q_off, kv_len, table, k_pages, v_pages, ctx=None, scale=SCALE):
    """All of out [L][n_q][hq][128] over rows [L][n_pages][P][8][128] of the values that are held.  q_off, kv_len: lists;
    ctx: (ctx_k, ctx_v [L][G][max_ctx][8][128], their lengths [layer][group], group of each sequence) or None.

    The bound is attend64's, and 2^-126 (1 + r max|v|) for r rows: many held values are 0, so an output may be a sum of weights near
    fp32's smallest normal number alone; a weight below that comes out as 0, and so may an output."""
    L, page, dev = out.shape[0], k_pages.shape[2], out.device
    worst, at = [], []
    for b, rows in enumerate(kv_len):
        n = q_off[b + 1] - q_off[b]
        if n == 0:
            continue
        r = torch.arange(max(rows, 0), device=dev)
        where = table[b].long()[r // page]
        k, v = k_pages[:, where, r % page], v_pages[:, where, r % page]
        seen = (r[None] <= rows - n + torch.arange(n, device=dev)[:, None]).expand(L, n, -1)
        if ctx is not None:
            ck, cv, lens, group = ctx
            c = torch.tensor([x[group[b]] for x in lens], device=dev)
            most = int(max(x[group[b]] for x in lens))
            k, v = (torch.cat([t[:, group[b], :most], y], 1) for t, y in ((ck, k), (cv, v)))
            mem = torch.arange(most, device=dev)[None] < c[:, None]
            seen = torch.cat([mem[:, None].expand(L, n, most), seen], 2)
        mine = slice(q_off[b], q_off[b + 1])
        ref, tol = attend64(q[:, mine], k, v, seen, scale, out.dtype)
        if k.shape[1]:
            tol = tol + 2.0 ** -126 * (1 + k.shape[1] * v.double().abs().amax())
        worst.append(((out[:, mine].double() - ref).abs() - tol).flatten(1).amax(1))   # not a number: stays one
        at += [(l, b) for l in range(L)]
    worst = torch.cat(worst).cpu().tolist()
    wrong = [(x, w) for x, w in zip(at, worst) if not w <= 0]
    assert not wrong, "%d of %d (layer, sequence) pairs are over their bound: %s" % (len(wrong), len(at), wrong[:6])
