"""Timed cases of the paged local cache: the append (norm, rotation, store) and the attention over
a shared memory context and the paged local rows.

A case is a batch of `groups` x `members` sequences.  The sequences of a group share one memory
context (and, where `prefix` is not 0, the first local pages: a question they all start from); each
has its own local rows behind that.  `tokens` are the new tokens of a call: every sequence brings
between `tokens_min` and `tokens` of them, ragged, and the packed arrays carry a few padding rows
behind the last sequence where `pad` is not 0.
"""
import math
import random

import numpy as np
import torch

own = False

HEADS, DIM = 8, 128
SCALE = 1.0 / math.sqrt(128.0)
EPS, THETA = 1e-6, 1e6


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
        # one query's decode step: its new row in all 18 layers at once, where launch latency is all
        _case("append", 18, 1, 1, 1, 1, 32, 0, 0, 64, 64, 64, "bf16", True, 0, 0, 0, 1, "append_one_token"),
        # a batch's decode step with sequences that have ended (no token) and padding rows
        _case("append", 18, 16, 16, 1, 0, 32, 0, 0, 2048, 1, 16, "bf16", True, 16, 7, 0, 2, "append_batch_step"),
        # the interleaved workload's prompts: 8 queries x 1,088 tokens, 18 layers
        _case("append", 18, 8, 1, 1088, 1088, 32, 0, 0, 0, 0, 64, "bf16", True, 16, 0, 0, 3, "append_prompts"),
        # long ragged chunks at far positions, keys that carry no norm, wide query heads
        _case("append", 2, 5, 1, 9001, 4099, 64, 0, 0, 5000, 1, 32, "bf16", False, 1 << 24, 1, 0, 4,
              "append_long_ragged"),
        # the 100M-token workload's decode: one query, ~4,300 memory rows and 64 local ones
        _case("attend", 18, 1, 1, 1, 1, 32, 4300, 0, 64, 64, 64, "f32", True, 0, 0, 0, 5, "attend_one_token"),
        # 16 samples of one question: memory and question shared, the answers their own
        _case("attend", 18, 1, 16, 1, 1, 32, 4300, 64, 512, 1, 64, "f32", True, 0, 0, 0, 6, "attend_samples"),
        # a serving step of one layer: 64 users with a memory each, one new token
        _case("attend", 1, 64, 1, 1, 0, 32, 4300, 0, 4000, 1, 16, "bf16", True, 0, 3, 0, 7, "attend_batch"),
        # 61 sequences behind one long shared prefix in pages, own tails
        _case("attend", 1, 1, 61, 1, 1, 64, 0, 30011, 700, 1, 128, "bf16", True, 0, 0, 0, 8, "attend_long_prefix"),
        # a mixed step: one sequence in ten brings a piece of its prompt, the others one token
        _case("attend", 2, 5, 6, 509, 1, 32, 1500, 100, 1024, 1, 32, "bf16", True, 0, 5, 10, 9, "attend_mixed"),
        # the interleaved workload's last round: 8 queries x 1,088 tokens over ~250 memory rows, 4 layers
        _case("attend", 4, 8, 1, 1088, 1088, 32, 250, 0, 0, 0, 64, "f32", True, 0, 0, 0, 10, "attend_prompts"),
        # one long prompt over its memory, a layer
        _case("attend", 1, 1, 1, 8000, 8000, 32, 4300, 0, 0, 0, 256, "bf16", True, 0, 0, 0, 11, "attend_long_prompt"),
        # both calls as a decode step makes them: append, then attend
        _case("step", 18, 2, 8, 1, 1, 32, 2200, 64, 512, 1, 64, "bf16", True, 16, 0, 0, 12, "step_samples"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "step"])
    kind = rng.choice(["one", "batch", "shared", "prompt", "mixed"])
    hq = rng.choice([8, 16, 32, 32, 64])
    page = rng.choice([16, 32, 64, 128, 256])
    out = rng.choice(["f32", "bf16"]) if op == "attend" else "bf16"
    norm, pad = rng.random() < 0.7, rng.choice([0, 0, 1, 6])
    far = rng.choice([0, 16, 1 << 20])
    ctx = rng.choice([0, _spread(rng, 1, 5000), _spread(rng, 200, 5000)])
    if op == "append":
        ctx = 0
    lengths = rng.randrange(1 << 20)
    if kind == "one":
        return _case(op, _spread(rng, 1, 18), 1, 1, 1, 1, hq, ctx, 0, _spread(rng, 1, 20000), 1, page, out, norm, far,
                     pad, 0, lengths)
    if kind == "batch":
        return _case(op, rng.choice([1, 2]), _spread(rng, 2, 48), 1, rng.choice([1, 1, 3]), rng.choice([0, 1]), hq,
                     ctx, 0, _spread(rng, 16, 4000), 1, page, out, norm, far, pad, 0, lengths)
    if kind == "shared":
        return _case(op, rng.choice([1, 2, 4]), rng.choice([1, 1, 2, 5]), _spread(rng, 2, 24), rng.choice([1, 1, 2]),
                     1, hq, ctx, _spread(rng, 1, 6000), _spread(rng, 1, 800), 1, page, out, norm, far, pad, 0, lengths)
    if kind == "prompt":
        tokens = _spread(rng, 17, 2000)
        return _case(op, 1, _spread(rng, 1, 3), 1, tokens, max(1, tokens // 2), min(hq, 32), ctx, 0,
                     _spread(rng, 1, 1500), 0, page, out, norm, far, pad, 0, lengths)
    return _case(op, 1, _spread(rng, 1, 4), rng.choice([1, 2, 5]), _spread(rng, 16, 600), 1, hq, ctx,
                 rng.choice([0, _spread(rng, 1, 2000)]), _spread(rng, 1, 1500), 1, page, out, norm, far, pad, 10,
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
    row = 2 * HEADS * DIM                        # bytes of one K or V row
    nbytes = flops = 0
    if case["op"] != "attend":
        nbytes += 2 * L * n * (2 * row + 2 * hq * DIM)
        flops += L * n * (HEADS + hq) * DIM * 6
    if case["op"] != "append":
        seen = kv = 0
        for g in range(case["groups"]):
            of = range(g * case["members"], (g + 1) * case["members"])
            live = any(new[b] for b in of)
            for l in range(L):
                kv += ctx[g][l] if live else 0
                seen += sum(new[b] * ctx[g][l] for b in of)
            kv += L * (pre[g] if live else 0)
            for b in of:
                kv += L * (rows[b] - pre[g] if new[b] else 0)
                seen += L * (new[b] * (rows[b] - new[b]) + new[b] * (new[b] + 1) // 2)
        nbytes += kv * 2 * row + L * n * hq * DIM * (2 + (4 if case["out"] == "f32" else 2))
        flops += seen * hq * DIM * 4
    return {"bytes": nbytes, "flops": flops}


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
    s = {"case": case, "max_new": max(new), "max_rows": max(rows), "max_ctx": max(max(c) for c in ctx),
         "q_off": i32(q_off.tolist()), "kv_len": i32(rows), "page_table": torch.from_numpy(table).to(dev),
         "pos_off": i32([host.randrange(case["far"] + 1) for _ in range(B)]),
         "grp_off": i32([M * g for g in range(G + 1)]), "pre_len": i32([p // P * P for p in pre]),
         "q": normal(L, n_q, hq, DIM, std=2.0),
         "k_pages": normal(L, n_pages, P, HEADS, DIM), "v_pages": normal(L, n_pages, P, HEADS, DIM)}
    if case["op"] != "attend":
        s["k_new"], s["v_new"] = normal(L, n_q, HEADS, DIM, std=1.5), normal(L, n_q, HEADS, DIM)
        s["q_out"] = torch.zeros_like(s["q"])
        s["w_k"] = (normal(L, DIM, std=0.25) + 1).to(bf16) if case["norm"] else None
        s["w_q"] = (normal(L, DIM, std=0.25) + 1).to(bf16) if case["norm"] else None
    if case["op"] != "append":
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
    msa.msa_paged_append(s["k_new"], s["v_new"], s["q"], s["q_off"], s["kv_len"], s["page_table"], s["k_pages"],
                         s["v_pages"], s["q_out"], EPS, THETA, pos_off=s["pos_off"], w_k=s["w_k"], w_q=s["w_q"])


def _attend_own(s, q):
    from routed_kv_memory_amd import msa
    if s["workspace"] is None:
        nbytes = msa.msa_paged_attend_workspace_size(q.shape[0], s["kv_len"].numel(), s["pre_len"].numel(),
                                                     q.shape[1], q.shape[2])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    msa.msa_paged_attend(q, s["q_off"], s["kv_len"], s["page_table"], s["k_pages"], s["v_pages"], SCALE, s["out"],
                         s["workspace"], grp_off=s["grp_off"], ctx_k=s["ctx_k"], ctx_v=s["ctx_v"],
                         ctx_len=s["ctx_len"] if s["ctx_k"] is not None else None, pre_len=s["pre_len"])


def _new_rows(s):
    """Of every packed token behind a sequence: its packed index, its sequence and its local row."""
    q_off, kv_len = s["q_off"].long(), s["kv_len"].long()
    t = torch.arange(s["q"].shape[1], device=q_off.device)
    t = t[t < q_off[-1]]
    b = torch.bucketize(t, q_off[1:], right=True)
    return t, b, kv_len[b] - q_off[b + 1] + t


def _turned(x, w, turn):
    """RMS norm per head (where w is given) and rotation of rows [L][n][heads][128], in 32 bits."""
    x = x.float()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()[:, None, None, :]
    a, b = x[..., :64], x[..., 64:]
    cos, sin = torch.cos(turn).float()[None, :, None, :], torch.sin(turn).float()[None, :, None, :]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append_plain(s):
    t, b, r = _new_rows(s)
    P = s["case"]["page"]
    # angles in 64 bits: those of far positions have lost their fraction in 32
    f = THETA ** (-torch.arange(64, device=t.device, dtype=torch.float64) / 64)
    turn = (s["pos_off"].long()[b] + r).double()[:, None] * f
    page = s["page_table"].long()[b, r // P]
    s["k_pages"][:, page, r % P] = _turned(s["k_new"][:, t], s["w_k"], turn).to(torch.bfloat16)
    s["v_pages"][:, page, r % P] = s["v_new"][:, t]
    s["q_out"][:, t] = _turned(s["q"][:, t], s["w_q"], turn).to(torch.bfloat16)


def _attend_plain(s, q):
    """Padded to [sequence][most tokens] and [sequence][memory rows + most local rows], masked softmax."""
    case, dev = s["case"], q.device
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
    k, v = s["k_pages"][:, pages, r % P], s["v_pages"][:, pages, r % P]       # [L][B][R][8][128]
    if C:
        k, v = torch.cat([s["ctx_k"][:, grp], k], 2), torch.cat([s["ctx_v"][:, grp], v], 2)
    x = q[:, at].float().reshape(L, B, T, HEADS, hq // HEADS, DIM).permute(0, 1, 3, 4, 2, 5)
    x = x.reshape(L, B, HEADS, hq // HEADS * T, DIM)
    sc = torch.matmul(x, k.float().permute(0, 1, 3, 4, 2)) * SCALE            # [L][B][8][heads x T][C + R]
    ok = r < (kv_len - new)[:, None, None] + i[:, None] + 1                   # [B][T][R]
    ok = ok[None].expand(L, B, T, R)
    if C:
        mem = torch.arange(C, device=dev) < s["ctx_len"].long()[:, grp, None]
        ok = torch.cat([mem[:, :, None].expand(L, B, T, C), ok], 3)
    sc = sc.view(L, B, HEADS, hq // HEADS, T, C + R).masked_fill_(~ok[:, :, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc = sc.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc.view(L, B, HEADS, hq // HEADS * T, C + R), v.float().permute(0, 1, 3, 2, 4))
    o = o.view(L, B, HEADS, hq // HEADS, T, DIM) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(L, B, T, hq, DIM)
    s["out"][:, at[live]] = o[:, live].to(s["out"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        if op != "attend":
            _append_own(s)
        if op != "append":
            _attend_own(s, s["q"] if op == "attend" else s["q_out"])
    else:
        if op != "attend":
            _append_plain(s)
        if op != "append":
            _attend_plain(s, s["q"] if op == "attend" else s["q_out"])
    if op == "append":
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q_out": s["q_out"]}
    if op == "attend":
        return {"out": s["out"]}
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q_out": s["q_out"], "out": s["out"]}


def _exact_turn(x, w, positions):
    """The rotation as a product of complex numbers, in 64 bits: x [n][heads][128], positions [n]."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / DIM + EPS) * w.double()
    f = torch.exp(torch.arange(64, device=x.device, dtype=torch.float64) * (-math.log(THETA) / 64))
    z = torch.complex(x[..., :64], x[..., 64:]) * torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                                                              positions.double()[:, None] * f)[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    P, op, L = case["page"], case["op"], case["layers"]
    ctx, _, new, rows = _lengths(case)
    table = s["page_table"].cpu().tolist()
    pos = s["pos_off"].cpu().tolist()
    starts = [sum(new[:b]) for b in range(len(new))]
    dev = s["q"].device
    # where each sequence's local rows lie among all rows of the cache
    spots = [torch.tensor([table[b][i // P] * P + i % P for i in range(rows[b])], dtype=torch.long, device=dev)
             for b in range(len(rows))]
    got = {}
    if op != "attend":
        kp, vp = s["k_pages"].double().flatten(1, 2), s["v_pages"].double().flatten(1, 2)
        qo = torch.zeros_like(s["q"], dtype=torch.float64)
        for l in range(L):
            for b, n in enumerate(new):
                if n == 0:
                    continue
                mine = slice(starts[b], starts[b] + n)
                p = torch.arange(rows[b] - n, rows[b], device=dev) + pos[b]
                kp[l, spots[b][rows[b] - n:]] = _exact_turn(s["k_new"][l, mine], None if s["w_k"] is None else s["w_k"][l], p)
                vp[l, spots[b][rows[b] - n:]] = s["v_new"][l, mine].double()
                qo[l, mine] = _exact_turn(s["q"][l, mine], None if s["w_q"] is None else s["w_q"][l], p)
        shape = s["k_pages"].shape
        got = {"k_pages": kp.view(shape), "v_pages": vp.view(shape), "q_out": qo}
        if op == "append":
            return got
        # what the cache and the rotated queries hold is rounded to their type before it is attended to
        s["k_pages"], s["v_pages"] = kp.to(torch.bfloat16).view(shape), vp.to(torch.bfloat16).view(shape)
        s["q"] = qo.to(torch.bfloat16)
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    g_heads = case["hq"] // HEADS
    for l in range(L):
        keys, values = s["k_pages"][l].flatten(0, 1), s["v_pages"][l].flatten(0, 1)
        for b, n in enumerate(new):
            if n == 0:
                continue
            g = b // case["members"]
            c = ctx[g][l]
            k, v = keys[spots[b]], values[spots[b]]
            if c:
                k, v = torch.cat([s["ctx_k"][l, g, :c], k]), torch.cat([s["ctx_v"][l, g, :c], v])
            hidden = torch.arange(rows[b], device=dev)[None] > torch.arange(rows[b] - n, rows[b], device=dev)[:, None]
            hidden = torch.nn.functional.pad(hidden, (c, 0))
            for h in range(HEADS):
                x = s["q"][l, starts[b]:starts[b] + n, h * g_heads:(h + 1) * g_heads].double().transpose(0, 1).contiguous()
                w = (x @ k[:, h].double().T.contiguous() * SCALE).masked_fill(hidden, -math.inf)
                w = torch.exp(w - torch.logsumexp(w, -1, keepdim=True))
                o = w @ v[:, h].double()
                out[l, starts[b]:starts[b] + n, h * g_heads:(h + 1) * g_heads] = o.transpose(0, 1)
    got["out"] = out
    return got
