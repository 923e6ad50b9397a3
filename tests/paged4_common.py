"""Shared by the tests of the paged local cache held in 4 bits: the format in 64 bits, written from its
definition, and batches whose pages hold it."""
import torch

from paged_common import Batch

ROW4 = 544
ELEMENTS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def exponents(m):
    """The smallest e with m <= 7 * 2^e, in [-125, 125], by trying all of them."""
    e = torch.arange(-125, 126, dtype=torch.float64, device=m.device)
    return (-125 + (m[..., None] > 7 * torch.exp2(e)).sum(-1)).clamp(max=125)


def quantise(x):
    """Rows x [..., 128] in 64 bits: codes [..., 128] and scale bytes [..., 4]."""
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
        codes, scales = quantise(rows)
        setattr(self, name + "4", pack(codes, scales))
        setattr(self, name, values(codes, scales).to(torch.bfloat16))

    def to_device(self):
        d = super().to_device()
        d["k_pages"], d["v_pages"] = self.k_pages4.to(self.device), self.v_pages4.to(self.device)
        return d
