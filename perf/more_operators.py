"""Timed cases of the paged local cache held in 4 bits: rows written and read back, rows read, and the
attention over a shared memory context and 4-bit local rows.

A block of 32 dims x of one head's row is held as e, the smallest whole number with max|x| <= 7 * 2^e (kept
in [-125, 125]), in a byte e + 127, and 32 codes: a sign and the index of the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
to |x| / 2^e (halfway: the even index; past 6: 6), two in a byte, the lower dim in the low half.  A page of P rows is [8
heads][P][64] bytes of codes and [8][P][4] of scales.  K is held as its value after norm and rotation is.

A case is a batch of `groups` x `members` sequences.  The sequences of a group share one memory
context (and, where `prefix` is not 0, the first local pages: a question they all start from); each
has its own local rows behind that.  `tokens` are the new tokens of a call (of "read": the rows that
are read): every sequence brings between `tokens_min` and `tokens` of them, ragged, and the packed
arrays carry a few padding rows behind the last sequence where `pad` is not 0.
"""
import math
import random

import numpy as np
import torch

own = False

HEADS, DIM = 8, 128
ROW4 = HEADS * (DIM // 2 + DIM // 32)            # bytes of a 4-bit row
SCALE = 1.0 / math.sqrt(128.0)
EPS, THETA = 1e-6, 1e6
EPS32 = float(np.float32(EPS))                   # the call takes floats


def _case(op, layers, groups, members, tokens, tokens_min, hq, ctx, prefix, local, local_min, page, out, norm, far,
          pad, mix, lengths, name=None):
    c = {"op": op, "layers": layers, "groups": groups, "members": members, "tokens": tokens,
         "tokens_min": tokens_min, "hq": hq, "ctx": ctx, "prefix": prefix, "local": local, "local_min": local_min,
         "page": page, "out": out, "norm": norm, "far": far, "pad": pad, "mix": mix, "lengths": lengths}
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one query's decode step: its new row in all 18 layers at once and read back, where latency is all
        _case("store", 18, 1, 1, 1, 1, 32, 0, 0, 64, 64, 64, "bf16", True, 0, 0, 0, 1, "store_one_token"),
        # a batch's decode step with sequences that have ended (no token) and padding rows
        _case("store", 18, 16, 16, 1, 0, 32, 0, 0, 2048, 1, 16, "bf16", True, 16, 7, 0, 2, "store_batch_step"),
        # the interleaved workload's prompts: 8 queries x 1,088 tokens, 18 layers
        _case("store", 18, 8, 1, 1088, 1088, 32, 0, 0, 0, 0, 64, "bf16", True, 16, 0, 0, 3, "store_prompts"),
        # long ragged chunks at far positions, keys that carry no norm, wide query heads
        _case("store", 2, 5, 1, 9001, 4099, 64, 0, 0, 5000, 1, 32, "bf16", False, 1 << 16, 1, 0, 4,
              "store_long_ragged"),
        # a short answer that becomes a memory document: its rows back in bf16
        _case("read", 18, 1, 1, 333, 333, 8, 0, 0, 0, 0, 64, "bf16", False, 0, 0, 0, 5, "read_answer"),
        # ended conversations of all lengths, read behind the question that is in the memory already
        _case("read", 18, 6, 1, 9000, 1, 8, 0, 0, 129, 0, 32, "bf16", False, 0, 3, 0, 6, "read_conversations"),
        # one query deep in a long conversation: ~4,300 memory rows, 32,000 local ones, all layers
        _case("attend", 18, 1, 1, 1, 1, 32, 4300, 0, 32000, 32000, 64, "f32", True, 0, 0, 0, 7, "attend_one_token"),
        # 16 samples of one question: memory and question shared, the answers their own
        _case("attend", 18, 1, 16, 1, 1, 32, 2200, 4000, 512, 1, 64, "f32", True, 0, 0, 0, 8, "attend_samples"),
        # a serving step of one layer: 64 users with a memory each, long conversations in small pages
        _case("attend", 1, 64, 1, 1, 0, 32, 1100, 0, 16000, 1, 16, "bf16", True, 0, 3, 0, 9, "attend_batch"),
        # five drafted tokens a sequence, checked at once
        _case("attend", 2, 24, 1, 5, 5, 64, 0, 0, 9000, 100, 32, "bf16", True, 0, 0, 0, 10, "attend_drafts"),
        # a mixed step: one sequence in ten brings a piece of its prompt, the others one token
        _case("attend", 2, 5, 6, 509, 1, 32, 1500, 100, 4096, 1, 32, "bf16", True, 0, 5, 10, 11, "attend_mixed"),
        # a piece of one long prompt: 4,000 tokens over its memory and the 28,000 rows before them, a layer
        _case("attend", 1, 1, 1, 4000, 4000, 32, 4300, 0, 28000, 28000, 256, "bf16", True, 0, 0, 0, 12,
              "attend_long_prompt"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend", "attend"])
    kind = rng.choice(["one", "batch", "prompt"] if op != "attend" else ["one", "batch", "shared", "prompt", "mixed"])
    hq = rng.choice([8, 16, 32, 32, 64])
    page = rng.choice([4, 16, 32, 64, 128, 512])
    out = rng.choice(["f32", "bf16"]) if op == "attend" else "bf16"
    norm, pad = rng.random() < 0.7, rng.choice([0, 0, 1, 6])
    far = rng.choice([0, 16, 1 << 16])
    ctx = rng.choice([0, _spread(rng, 1, 5000), _spread(rng, 200, 5000)]) if op == "attend" else 0
    lengths = rng.randrange(1 << 20)
    if kind == "one":
        tokens = _spread(rng, 1, 4000) if op == "read" else 1
        return _case(op, _spread(rng, 1, 18), 1, 1, tokens, tokens, hq, ctx, 0, _spread(rng, 1, 40000), 1, page, out,
                     norm, far, pad, 0, lengths)
    if kind == "batch":
        return _case(op, rng.choice([1, 2]), _spread(rng, 2, 48), 1, rng.choice([1, 1, 3, 7]), rng.choice([0, 1]), hq,
                     ctx, 0, _spread(rng, 16, 12000), 1, page, out, norm, far, pad, 0, lengths)
    if kind == "shared":
        return _case(op, rng.choice([1, 2, 4]), rng.choice([1, 1, 2, 5]), _spread(rng, 2, 16), rng.choice([1, 1, 2]),
                     1, hq, ctx, _spread(rng, 1, 9000), _spread(rng, 1, 800), 1, page, out, norm, far, pad, 0, lengths)
    if kind == "prompt":
        tokens = _spread(rng, 17, 2000)
        return _case(op, 1, _spread(rng, 1, 3), 1, tokens, max(1, tokens // 2), min(hq, 32), ctx, 0,
                     _spread(rng, 1, 6000), 0, page, out, norm, far, pad, 0, lengths)
    return _case(op, 1, _spread(rng, 1, 4), rng.choice([1, 2, 5]), _spread(rng, 16, 600), 1, hq, ctx,
                 rng.choice([0, _spread(rng, 1, 2000)]), _spread(rng, 1, 5000), 1, page, out, norm, far, pad, 10,
                 lengths)


def _lengths(case):
    """Per group: memory rows and shared local rows; per sequence: new tokens and all local rows."""
    rng = random.Random(case["lengths"])
    ctx, pre, new, rows = [], [], [], []
    for g in range(case["groups"]):
        ctx.append([rng.randint(case["ctx"] - case["ctx"] // 8, case["ctx"]) for _ in range(case["layers"])])
        pre.append(rng.randint(case["prefix"] - case["prefix"] // 8, case["prefix"]))
        for m in range(case["members"]):
            n = rng.randint(case["tokens_min"], case["tokens"])
            if case["mix"]:     # one sequence in `mix` brings a piece of a prompt, the others one token
                n = case["tokens"] if len(new) % case["mix"] == case["mix"] // 3 else 1
            n = n if new else max(1, n)          # a call has one token at least
            new.append(n)
            rows.append(pre[-1] + n + (rng.randint(case["local_min"], case["local"]) if case["local"] else 0))
    return ctx, pre, new, rows


def work(case):
    ctx, pre, new, rows = _lengths(case)
    L, hq, n = case["layers"], case["hq"], sum(new)
    row = 2 * HEADS * DIM                        # bytes of one bf16 K or V row
    if case["op"] == "read":
        return {"bytes": L * n * 2 * (ROW4 + row), "flops": L * n * 2 * HEADS * DIM}
    if case["op"] == "store":                    # the rows that were written are read back
        return {"bytes": L * n * (2 * row + 2 * 2 * hq * DIM + 2 * ROW4 + 2 * (ROW4 + row)),
                "flops": L * n * (4 * HEADS + hq) * DIM * 6}
    nbytes = seen = 0
    for g in range(case["groups"]):
        of = range(g * case["members"], (g + 1) * case["members"])
        live = any(new[b] for b in of)
        for l in range(L):
            nbytes += ctx[g][l] * 2 * row if live else 0
            seen += sum(new[b] * ctx[g][l] for b in of)
        nbytes += L * (pre[g] if live else 0) * 2 * ROW4
        for b in of:
            nbytes += L * (rows[b] - pre[g] if new[b] else 0) * 2 * ROW4
            seen += L * (new[b] * (rows[b] - new[b]) + new[b] * (new[b] + 1) // 2)
    nbytes += L * n * hq * DIM * (2 + (4 if case["out"] == "f32" else 2))
    return {"bytes": nbytes, "flops": seen * hq * DIM * 4}


def _two_to(e, like):
    """2^e in the type of `like`, exactly; |e| at most 126."""
    if like.dtype == torch.float64:
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _held(x):
    """Rows [..., 128] as they are held: codes [..., 64] and scales [..., 4] bytes."""
    x = x.unflatten(-1, (4, 32))
    mant, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = torch.where(mant == 0, -125, e - torch.where(mant <= 0.875, 3, 2)).clamp(-125, 125)
    y = x.abs() * _two_to(-e, x)
    code = ((y > 0.25).byte() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5))
    code = (code + 8 * torch.signbit(x)).byte().flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).byte().squeeze(-1)


def _parts(pages, P):
    """Pages [L][n_pages][544 P] as codes [L][n_pages][P][8][64] and scales [L][n_pages][P][8][4]."""
    codes = pages[..., :512 * P].unflatten(-1, (HEADS, P, DIM // 2)).transpose(2, 3)
    return codes, pages[..., 512 * P:].unflatten(-1, (HEADS, P, DIM // 32)).transpose(2, 3)


def _values(codes, scales):
    """What codes [..., 64] and scales [..., 4] stand for, in 32 bits [..., 128]."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    one = torch.cat([one, -one])
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([one[byte & 15], one[byte >> 4]], -1)                 # of a byte
    x = pair[codes.int()].flatten(-2).unflatten(-1, (4, 32))
    return (x * (scales.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    ctx, pre, new, rows = _lengths(case)
    L, G, M, hq, P = case["layers"], case["groups"], case["members"], case["hq"], case["page"]
    B = G * M
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).mul_(std).to(bf16)

    def cache(n_pages):
        """Pages that rows of normal values were written to."""
        pages = torch.empty(L, n_pages, ROW4 * P, dtype=torch.uint8, device=dev)
        codes, scales = _parts(pages, P)
        step = max(1, (1 << 15) // P)
        for l in range(L):
            for at in range(0, n_pages, step):
                n = min(step, n_pages - at)
                codes[l, at:at + n], scales[l, at:at + n] = _held(normal(n, P, HEADS, DIM).float())
        return pages

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    # pages: the group's shared ones first, then each sequence's own (a page that the prefix ends in is
    # a sequence's own from there on, so it shares only whole pages)
    pages = []
    used = 0
    for b in range(B):
        whole = pre[b // M] // P
        mine = -(-rows[b] // P)
        if b % M == 0:
            shared = list(range(used, used + whole))
            used += whole
        pages.append(shared + list(range(used, used + mine - whole)))
        used += mine - whole
    n_pages = max(1, used) + 3
    order = list(range(n_pages))
    host.shuffle(order)                          # a served cache is fragmented
    max_pages = max(1, max(len(p) for p in pages))
    table = np.zeros((B, max_pages), np.int32)
    for b, p in enumerate(pages):
        table[b, :len(p)] = [order[i] for i in p]
    n_q = sum(new) + case["pad"]
    q_off = np.concatenate([[0], np.cumsum(new)])
    s = {"case": case, "max_new": max(new), "max_rows": max(rows), "max_ctx": max(max(c) for c in ctx), "n_q": n_q,
         "q_off": i32(q_off.tolist()), "kv_len": i32(rows), "page_table": torch.from_numpy(table).to(dev),
         "pos_off": i32([host.randrange(case["far"] + 1) for _ in range(B)]),
         "row0": i32([r - n for r, n in zip(rows, new)]),
         "grp_off": i32([M * g for g in range(G + 1)]), "pre_len": i32([p // P * P for p in pre]),
         "k_pages": cache(n_pages), "v_pages": cache(n_pages)}
    if case["op"] != "read":
        s["q"] = normal(L, n_q, hq, DIM, std=2.0)
    if case["op"] != "attend":
        s["k_out"], s["v_out"] = (torch.zeros(L, n_q, HEADS, DIM, device=dev, dtype=bf16) for _ in range(2))
    if case["op"] == "store":
        s["k_new"], s["v_new"] = normal(L, n_q, HEADS, DIM, std=1.5), normal(L, n_q, HEADS, DIM)
        s["q_out"] = torch.zeros_like(s["q"])
        s["w_k"] = (normal(L, DIM, std=0.25) + 1).to(bf16) if case["norm"] else None
        s["w_q"] = (normal(L, DIM, std=0.25) + 1).to(bf16) if case["norm"] else None
    if case["op"] == "attend":
        C = s["max_ctx"]
        s["ctx_len"] = i32([[ctx[g][l] for g in range(G)] for l in range(L)])
        s["ctx_k"] = normal(L, G, C, HEADS, DIM) if C else None
        s["ctx_v"] = normal(L, G, C, HEADS, DIM) if C else None
        s["out"] = torch.zeros(L, n_q, hq, DIM, device=dev,
                               dtype=torch.float32 if case["out"] == "f32" else bf16)
        s["workspace"] = None                    # allocated by the first call, kept for the next ones
    return s


def _append_own(s):
    from routed_kv_memory_amd import msa
    msa.msa_paged_append4(s["k_new"], s["v_new"], s["q"], s["q_off"], s["kv_len"], s["page_table"], s["k_pages"],
                          s["v_pages"], s["q_out"], EPS, THETA, pos_off=s["pos_off"], w_k=s["w_k"], w_q=s["w_q"])


def _read_own(s):
    from routed_kv_memory_amd import msa
    msa.msa_paged_read4(s["k_pages"], s["v_pages"], s["q_off"], s["page_table"], s["k_out"], s["v_out"],
                        row0=s["row0"])


def _attend_own(s):
    from routed_kv_memory_amd import msa
    q = s["q"]
    if s["workspace"] is None:
        nbytes = msa.msa_paged_attend4_workspace_size(q.shape[0], s["kv_len"].numel(), s["pre_len"].numel(),
                                                      q.shape[1], q.shape[2])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    msa.msa_paged_attend4(q, s["q_off"], s["kv_len"], s["page_table"], s["k_pages"], s["v_pages"], SCALE, s["out"],
                          s["workspace"], grp_off=s["grp_off"], ctx_k=s["ctx_k"], ctx_v=s["ctx_v"],
                          ctx_len=s["ctx_len"] if s["ctx_k"] is not None else None, pre_len=s["pre_len"])


def _new_rows(s):
    """Of every packed token behind a sequence: its packed index, its sequence and its local row."""
    q_off, row0 = s["q_off"].long(), s["row0"].long()
    t = torch.arange(s["n_q"], device=q_off.device)
    t = t[t < q_off[-1]]
    b = torch.bucketize(t, q_off[1:], right=True)
    return t, b, row0[b] + t - q_off[b]


def _turned(x, w, turn):
    """RMS norm per head (where w is given) and rotation of rows [L][n][heads][128], in the type of x."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS32) * w.to(x.dtype)[:, None, None, :]
    a, b = x[..., :64], x[..., 64:]
    cos, sin = torch.cos(turn).to(x.dtype)[None, :, None, :], torch.sin(turn).to(x.dtype)[None, :, None, :]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append_plain(s):
    t, b, r = _new_rows(s)
    P = s["case"]["page"]
    # angles in 64 bits: those of far positions have lost their fraction in 32
    f = THETA ** (-torch.arange(64, device=t.device, dtype=torch.float64) / 64)
    turn = (s["pos_off"].long()[b] + r).double()[:, None] * f
    page = s["page_table"].long()[b, r // P]
    # keys in 64 bits: a value next to a border of two codes falls to either side of it in 32
    for pages, x in ((s["k_pages"], _turned(s["k_new"][:, t].double(), s["w_k"], turn)),
                     (s["v_pages"], s["v_new"][:, t].float())):
        codes, scales = _parts(pages, P)
        codes[:, page, r % P], scales[:, page, r % P] = _held(x)
    s["q_out"][:, t] = _turned(s["q"][:, t].float(), s["w_q"], turn).to(torch.bfloat16)


def _read_plain(s):
    t, b, r = _new_rows(s)
    P = s["case"]["page"]
    page = s["page_table"].long()[b, r // P]
    for pages, out in ((s["k_pages"], s["k_out"]), (s["v_pages"], s["v_out"])):
        codes, scales = _parts(pages, P)
        out[:, t] = _values(codes[:, page, r % P], scales[:, page, r % P]).to(torch.bfloat16)


def _attend_plain(s):
    """Padded to [sequence][most tokens] and [sequence][memory rows + most local rows], masked softmax."""
    case, q = s["case"], s["q"]
    dev = q.device
    L, hq, P, T, C, R = case["layers"], case["hq"], case["page"], s["max_new"], s["max_ctx"], s["max_rows"]
    B = case["groups"] * case["members"]
    q_off, kv_len = s["q_off"].long(), s["kv_len"].long()
    new = q_off[1:] - q_off[:-1]
    i = torch.arange(T, device=dev)
    at = (q_off[:-1, None] + i).clamp(max=q.shape[1] - 1)                     # [B][T]
    live = i < new[:, None]
    r = torch.arange(R, device=dev)
    pages = s["page_table"].long()[:, (r // P).clamp(max=s["page_table"].shape[1] - 1)]
    grp = torch.arange(B, device=dev) // case["members"]

    def rows(pages4, ctx):
        codes, scales = _parts(pages4, P)
        x = _values(codes[:, pages, r % P], scales[:, pages, r % P])           # [L][B][R][8][128]
        return torch.cat([ctx[:, grp].float(), x], 2) if C else x

    x = q[:, at].float().reshape(L, B, T, HEADS, hq // HEADS, DIM).permute(0, 1, 3, 4, 2, 5)
    x = x.reshape(L, B, HEADS, hq // HEADS * T, DIM)
    sc = torch.matmul(x, rows(s["k_pages"], s["ctx_k"]).permute(0, 1, 3, 4, 2)) * SCALE   # [L][B][8][heads x T][C + R]
    ok = r < (kv_len - new)[:, None, None] + i[:, None] + 1                   # [B][T][R]
    ok = ok[None].expand(L, B, T, R)
    if C:
        mem = torch.arange(C, device=dev) < s["ctx_len"].long()[:, grp, None]
        ok = torch.cat([mem[:, :, None].expand(L, B, T, C), ok], 3)
    sc = sc.view(L, B, HEADS, hq // HEADS, T, C + R).masked_fill_(~ok[:, :, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc = sc.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = sc.sum(-1, keepdim=True)
    v = rows(s["v_pages"], s["ctx_v"])
    o = torch.matmul(sc.view(L, B, HEADS, hq // HEADS * T, C + R), v.permute(0, 1, 3, 2, 4))
    o = o.view(L, B, HEADS, hq // HEADS, T, DIM) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(L, B, T, hq, DIM)
    s["out"][:, at[live]] = o[:, live].to(s["out"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "store":
            _append_own(s)
        if op == "attend":
            _attend_own(s)
        else:
            _read_own(s)
    else:
        if op == "store":
            _append_plain(s)
        if op == "attend":
            _attend_plain(s)
        else:
            _read_plain(s)
    if op == "attend":
        return {"out": s["out"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"k": s["k_out"], "v": s["v_out"], "q_out": s["q_out"]}


def _exact_turn(x, w, positions):
    """The rotation as a product of complex numbers, in 64 bits: x [n][heads][128], positions [n]."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / DIM + EPS32) * w.double()
    f = torch.exp(torch.arange(64, device=x.device, dtype=torch.float64) * (-math.log(THETA) / 64))
    z = torch.complex(x[..., :64], x[..., 64:]) * torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                                                              positions.double()[:, None] * f)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_rounded(x):
    """Each block of 32 of x [..., 128] (64 bits) rounded to what 4 bits and its power of two can say."""
    b = x.reshape(*x.shape[:-1], 4, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 7)), torch.full_like(top, -125)).clamp(-125, 125)
    unit = torch.exp2(e)
    y = b / unit
    a = y.abs()
    step = torch.where(a <= 2, 0.5, torch.where(a <= 4, 1.0, 2.0))             # between neighbours there
    return (torch.clamp(torch.round(y / step) * step, -6, 6) * unit).reshape(x.shape)


def _exact_rows(pages, P, spots):
    """Rows of a layer's pages [n_pages][544 P] in 64 bits, [n][8][128]; spots: page, row in it."""
    page, row = spots
    n = page.shape[0]
    head = torch.arange(HEADS, device=pages.device)[None, :, None]
    flat = (page * (ROW4 * P))[:, None, None]
    codes = pages.flatten()[flat + (head * P + row[:, None, None]) * 64 + torch.arange(64, device=pages.device)]
    power = pages.flatten()[flat + 512 * P + (head * P + row[:, None, None]) * 4 + torch.arange(4, device=pages.device)]
    c = torch.stack([codes % 16, codes // 16], -1).reshape(n, HEADS, DIM).long()
    m = c % 8                                       # two bits of exponent, one of fraction
    x = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * torch.exp2((m // 2 - 1).double()))
    x = torch.where(c >= 8, -x, x).reshape(n, HEADS, 4, 32) * torch.exp2(power.double() - 127)[..., None]
    return x.reshape(n, HEADS, DIM)


def exact(case, seed):
    s = prepare(case, seed)
    P, op, L = case["page"], case["op"], case["layers"]
    ctx, _, new, rows = _lengths(case)
    table = s["page_table"].long()
    pos = s["pos_off"].cpu().tolist()
    starts = [sum(new[:b]) for b in range(len(new))]
    dev = table.device

    def spots(b, first, end):
        r = torch.arange(first, end, device=dev)
        return table[b, r // P], r % P

    if op != "attend":
        got = {n: torch.zeros_like(s[k], dtype=torch.float64)
               for n, k in (("k", "k_out"), ("v", "v_out"), ("q_out", "q_out")) if k in s}
        for l in range(L):
            for b, n in enumerate(new):
                if n == 0:
                    continue
                mine = slice(starts[b], starts[b] + n)
                if op == "read":
                    where = spots(b, rows[b] - n, rows[b])
                    got["k"][l, mine] = _exact_rows(s["k_pages"][l], P, where)
                    got["v"][l, mine] = _exact_rows(s["v_pages"][l], P, where)
                    continue
                p = torch.arange(rows[b] - n, rows[b], device=dev) + pos[b]
                w = lambda x: None if x is None else x[l]
                got["k"][l, mine] = _exact_rounded(_exact_turn(s["k_new"][l, mine], w(s["w_k"]), p))
                got["v"][l, mine] = _exact_rounded(s["v_new"][l, mine].double())
                got["q_out"][l, mine] = _exact_turn(s["q"][l, mine], w(s["w_q"]), p)
        return got
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    g_heads = case["hq"] // HEADS
    for l in range(L):
        for b, n in enumerate(new):
            if n == 0:
                continue
            g = b // case["members"]
            c = ctx[g][l]
            where = spots(b, 0, rows[b])
            k, v = _exact_rows(s["k_pages"][l], P, where), _exact_rows(s["v_pages"][l], P, where)
            if c:
                k, v = torch.cat([s["ctx_k"][l, g, :c].double(), k]), torch.cat([s["ctx_v"][l, g, :c].double(), v])
            hidden = torch.arange(rows[b], device=dev)[None] > torch.arange(rows[b] - n, rows[b], device=dev)[:, None]
            hidden = torch.nn.functional.pad(hidden, (c, 0))
            for h in range(HEADS):
                x = s["q"][l, starts[b]:starts[b] + n, h * g_heads:(h + 1) * g_heads].double().transpose(0, 1).contiguous()
                w = (x @ k[:, h].T.contiguous() * SCALE).masked_fill(hidden, -math.inf)
                w = torch.exp(w - torch.logsumexp(w, -1, keepdim=True))
                o = w @ v[:, h].contiguous()
                out[l, starts[b]:starts[b] + n, h * g_heads:(h + 1) * g_heads] = o.transpose(0, 1)
    return {"out": out}
