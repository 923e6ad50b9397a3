"""Attention over paged rows in 64 bits on the GPU, for batches whose every token is looked at."""
import math

import torch

SCALE = 1.0 / math.sqrt(128.0)
BF16 = torch.bfloat16


def attend64(q, k, v, seen, scale, dtype):
    """In each layer, tokens q [L][n][hq][128] over rows k, v [L][r][8][128], of which token i sees those of
    seen [L][n][r]: (out [L][n][hq][128], how far off a kernel may be).

    With u = 2^-24 (half an fp32 step): a score is a sum of 128 exact products, fewer than 16 roundings on any
    path, so off by at most 16 u sum |q k| scale; its distance to the maximum adds a few roundings of at most the
    scores' spread (2^-22 of it).  exp2 is right to one step (2^-23), three bf16 parts hold all but 2^-25 of a
    weight: 2^-22 together; one bf16 value (bf16 output) is off by half its step, 2^-8.  Sums over r rows: at
    most r u.  A relative error d of every weight moves the output by at most 2 d sum w |v|."""
    L, n, hq, r, G = *q.shape[:3], k.shape[1], q.shape[2] // 8
    if r == 0:
        z = torch.zeros(L, n, hq, 128, dtype=torch.float64, device=q.device)
        return z, z
    x = q.double().view(L, n, 8, G, 128).permute(0, 2, 1, 3, 4).reshape(L, 8, n * G, 128)
    kt = k.double().permute(0, 2, 3, 1).contiguous()
    vh = v.double().permute(0, 2, 1, 3).contiguous()
    seen = seen.repeat_interleave(G, 1)[:, None]                                  # [L][1][n G][r]
    some = seen.any(-1, keepdim=True)
    s = torch.matmul(x, kt) * scale
    big = (torch.matmul(x.abs(), kt.abs()) * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
    low = torch.where(some, s.masked_fill(~seen, math.inf).amin(-1, keepdim=True), 0.0)
    s = s.masked_fill(~seen, -math.inf)
    top = torch.where(some, s.amax(-1, keepdim=True), 0.0)
    w = torch.exp(s - top)
    w = w / torch.where(some, w.sum(-1, keepdim=True), 1.0)
    out, mass = torch.matmul(w, vh), torch.matmul(w, vh.abs())
    u = 2.0 ** -24
    d = 16 * u * big + 2.0 ** -22 * (top - low + 8) + 2.0 ** -22 + r * u
    if dtype == BF16:
        d = d + 2.0 ** -8
    tol = 2 * d * mass
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * (out.abs() + tol)
    back = lambda t: t.view(L, 8, n, G, 128).permute(0, 2, 1, 3, 4).reshape(L, n, hq, 128)
    return back(out), back(tol)


def check_every_token(out, q, q_off, kv_len, table, k_pages, v_pages, ctx=None, scale=SCALE):
    """All of out [L][n_q][hq][128].  q_off, kv_len: lists; ctx: (ctx_k, ctx_v [L][G][max_ctx][8][128], their
    lengths [layer][group], group of each sequence) or None.  The rest as the call takes it."""
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
        worst.append(((out[:, mine].double() - ref).abs() - tol).flatten(1).amax(1))   # not a number: stays one
        at += [(l, b) for l in range(L)]
    worst = torch.cat(worst).cpu().tolist()
    wrong = [(x, w) for x, w in zip(at, worst) if not w <= 0]
    assert not wrong, "%d of %d (layer, sequence) pairs are over their bound: %s" % (len(wrong), len(at), wrong[:6])
