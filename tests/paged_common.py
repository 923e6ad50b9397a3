"""Shared by the tests of the paged local cache: batches with random pages, and the append and the
attention in 64 bits, written from their formulas."""
import math

import numpy as np
import torch

EPS, THETA = 1e-6, 1e6
SCALE = 1.0 / math.sqrt(128.0)
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2      # half a step, relative to the value


class Batch:
    """groups: number of sequences of each group (None: every sequence its own).  new, rows: new
    tokens and local rows (new ones included) of each sequence.  ctx: memory rows [layer][group] or
    None.  pre: shared local rows of each group or None; a group's sequences share the pages that
    hold these rows.  Page numbers are shuffled and the pool has spare pages."""

    def __init__(self, new, rows, *, groups=None, ctx=None, pre=None, page=16, hq=32, layers=1, pad=0, seed=0,
                 q_std=1.0, max_ctx=None, device="cuda"):
        self.new, self.rows, self.page, self.hq, self.L, self.pad = list(new), list(rows), page, hq, layers, pad
        self.B = len(self.new)
        self.groups = [1] * self.B if groups is None else list(groups)
        self.G = len(self.groups)
        self.grp_off = np.concatenate([[0], np.cumsum(self.groups)]).astype(int).tolist()
        self.group_of = [g for g, n in enumerate(self.groups) for _ in range(n)]
        self.q_off = np.concatenate([[0], np.cumsum(self.new)]).astype(int).tolist()
        self.n_q = self.q_off[-1] + pad
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.pre = pre
        used, tables = 0, []
        for b in range(self.B):
            g = self.group_of[b]
            first = self.grp_off[g]
            whole = 0 if pre is None or b == first else min(-(-pre[g] // page), len(tables[first]))
            need = max(0, -(-self.rows[b] // page))
            mine = (tables[first][:whole] if whole else [])[:need]
            fresh = need - len(mine)
            tables.append(mine + list(range(used, used + fresh)))
            used += fresh
        self.n_pages = used + 3
        order = rng.permutation(self.n_pages)
        self.max_pages = max(1, max((len(t) for t in tables), default=1))
        self.table = np.full((self.B, self.max_pages), int(order[-1]), np.int32)
        for b, t in enumerate(tables):
            self.table[b, :len(t)] = order[t]

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=gen).mul_(std).to(torch.bfloat16)

        L = layers
        self.q = normal(L, self.n_q, hq, 128, std=q_std)
        self.k_new, self.v_new = normal(L, self.n_q, 8, 128), normal(L, self.n_q, 8, 128)
        self.w_k = (normal(L, 128, std=0.25) + 1).to(torch.bfloat16)
        self.w_q = (normal(L, 128, std=0.25) + 1).to(torch.bfloat16)
        self.k_pages, self.v_pages = normal(L, self.n_pages, page, 8, 128), normal(L, self.n_pages, page, 8, 128)
        self.ctx = ctx
        self.ctx_k = self.ctx_v = None
        if ctx is not None:
            self.max_ctx = max_ctx or max(1, max(max(c) for c in ctx))
            self.ctx_k, self.ctx_v = normal(L, self.G, self.max_ctx, 8, 128), normal(L, self.G, self.max_ctx, 8, 128)
        self.device = device

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.device)

    def to_device(self):
        """The arrays as the calls take them."""
        d = lambda t: None if t is None else t.to(self.device)
        return {"q": d(self.q), "k_new": d(self.k_new), "v_new": d(self.v_new), "w_k": d(self.w_k), "w_q": d(self.w_q),
                "k_pages": d(self.k_pages), "v_pages": d(self.v_pages), "ctx_k": d(self.ctx_k),
                "ctx_v": d(self.ctx_v), "ctx_len": None if self.ctx is None else self.i32(self.ctx),
                "q_off": self.i32(self.q_off), "kv_len": self.i32(self.rows),
                "page_table": torch.from_numpy(self.table).to(self.device),
                "grp_off": None if self.groups == [1] * self.B else self.i32(self.grp_off),
                "pre_len": None if self.pre is None else self.i32(self.pre)}

    def spot(self, b, r):
        """Page and row in it of sequence b's local row r."""
        return int(self.table[b, r // self.page]), r % self.page

    def local(self, pages, layer, b, n):
        """Sequence b's first n local rows [n][8][128]."""
        if n <= 0:
            return pages.new_zeros((0, 8, 128))
        r = torch.arange(n)
        t = torch.from_numpy(self.table[b].astype(np.int64))
        return pages[layer, t[r // self.page], r % self.page]


def turned(x, w, positions, eps=EPS, theta=THETA):
    """Rows x [n][heads][128], normed per head (w [128] or None) and turned, in 64 bits; and the
    largest sum of the two products behind each value (what the rounding errors are relative to)."""
    theta, eps = float(np.float32(theta)), float(np.float32(eps))     # the calls take floats
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    f = torch.tensor([theta ** (-e / 64.0) for e in range(64)], dtype=torch.float64)
    angle = torch.as_tensor(positions, dtype=torch.float64)[:, None] * f
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :64], x[..., 64:]
    size = a.abs() + b.abs()
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([size, size], -1)


def attention(b: Batch, layer, seq, i, k_pages=None, v_pages=None, q=None, scale=SCALE, bf16=False):
    """Token i of a sequence in 64 bits: (out [hq][128], how far off a kernel may be).

    Bound of the error: scores are sums of 128 products in fp32 (fewer than 16 roundings on any path
    through the sum), so a score is off by at most 16 * 2^-24 * sum |q k| * scale, plus a rounding of
    its difference to the maximum; exp and the product with V add 2^-17 (16 significant bits of each
    probability; half a bf16 step with bf16 output); sums over n rows in fp32 at most n * 2^-24.  A
    relative error d of every weight moves the output by at most 2 d sum w |v|."""
    k_pages = b.k_pages if k_pages is None else k_pages
    v_pages = b.v_pages if v_pages is None else v_pages
    q = b.q if q is None else q
    vis = max(0, b.rows[seq] - b.new[seq] + i + 1)
    k, v = b.local(k_pages, layer, seq, vis), b.local(v_pages, layer, seq, vis)
    g = b.group_of[seq]
    if b.ctx is not None:
        c = b.ctx[layer][g]
        k, v = torch.cat([b.ctx_k[layer, g, :c], k]), torch.cat([b.ctx_v[layer, g, :c], v])
    n = k.shape[0]
    if n == 0:
        z = torch.zeros(b.hq, 128, dtype=torch.float64)
        return z, z
    x = q[layer, b.q_off[seq] + i].double().view(8, b.hq // 8, 128)
    k, v = k.double().permute(1, 0, 2), v.double().permute(1, 0, 2)             # [8][n][128]
    s = torch.matmul(x, k.transpose(1, 2).contiguous()) * scale
    big = (torch.matmul(x.abs(), k.abs().transpose(1, 2).contiguous()) * scale).amax(-1, keepdim=True)
    w = torch.softmax(s, -1)
    out = torch.matmul(w, v)
    mass = torch.matmul(w, v.abs())
    spread = (s.amax(-1, keepdim=True) - s.amin(-1, keepdim=True)) + 8
    d = 16 * 2.0 ** -24 * big + 2.0 ** -22 * spread + 2.0 ** -17 + n * 2.0 ** -24
    if bf16:
        d = d + HALF_BF16
    tol = 2 * d * mass
    if bf16:
        tol = tol + HALF_BF16 * (out.abs() + tol)
    return out.reshape(b.hq, 128), tol.reshape(b.hq, 128)


def check_attention(b: Batch, out, tokens=None, k_pages=None, v_pages=None, q=None, scale=SCALE):
    """Every new token (or those given as (layer, seq, i)) of out [L][n_q][hq][128] against 64 bits."""
    bf16 = out.dtype == torch.bfloat16
    got = out.detach().cpu().double()
    if tokens is None:
        tokens = [(l, s, i) for l in range(b.L) for s in range(b.B) for i in range(b.new[s])]
    for l, s, i in tokens:
        ref, tol = attention(b, l, s, i, k_pages, v_pages, q, scale, bf16)
        x = got[l, b.q_off[s] + i]
        assert torch.isfinite(x).all(), (l, s, i)
        over = ((x - ref).abs() - tol).max().item()
        assert over <= 0, "layer %d sequence %d token %d: %g over its bound" % (l, s, i, over)
