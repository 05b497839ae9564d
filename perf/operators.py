"""Cases of the serving operators that stand between the weight-only products of a decode step: writing keys and
values into a paged 8-bit cache, reading them back, attention over that cache, and the choice of the next token.

Every case is a dict of plain values; `prepare` makes what a program holds before the call, `run` makes one pass,
either in plain torch operations (`own` false) or through this package (`own` true), and `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"int8": 127.0, "e4m3": 448.0}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a served batch: one new token for each of 64 sequences
        dict(name="write_step", op="write", fmt="int8", dtype="bf16", order="hsd", batch=64, heads=8, d=128, page=64,
             len_lo=60, len_hi=4000, new_lo=1, new_hi=1),
        # prompts of odd lengths entering the cache, in the type the weight-only products return
        dict(name="write_prompt", op="write", fmt="e4m3", dtype="fp32", order="hsd", batch=8, heads=8, d=128, page=64,
             len_lo=1001, len_hi=4093, new_lo=1001, new_hi=4093),
        # a short sequence read back whole
        dict(name="read_short", op="read", fmt="int8", dtype="fp32", order="shd", batch=1, heads=8, d=128, page=16,
             len_lo=513, len_hi=513, new_lo=513, new_hi=513),
        # long prefixes moved out of the cache
        dict(name="read_long", op="read", fmt="e4m3", dtype="bf16", order="hsd", batch=4, heads=8, d=128, page=128,
             len_lo=20001, len_hi=32768, new_lo=20001, new_hi=32768),
        # one user, a conversation of about a thousand tokens: latency
        dict(name="attn_one", op="attn", fmt="int8", dtype="bf16", order="hsd", batch=1, heads=8, group=4, d=128,
             page=64, len_lo=1003, len_hi=1003, new_lo=1, new_hi=1, window=0),
        # a served batch of ragged lengths, one token each
        dict(name="attn_batch", op="attn", fmt="int8", dtype="bf16", order="hsd", batch=64, heads=8, group=4, d=128,
             page=64, len_lo=300, len_hi=8192, new_lo=1, new_hi=1, window=0),
        # two very long contexts with a wide group of query heads
        dict(name="attn_long", op="attn", fmt="e4m3", dtype="fp16", order="shd", batch=2, heads=8, group=8, d=128,
             page=128, len_lo=100001, len_hi=131072, new_lo=1, new_hi=1, window=0),
        # prompt chunks of 2048 tokens against caches of up to 8192
        dict(name="attn_prompt", op="attn", fmt="int8", dtype="bf16", order="hsd", batch=4, heads=8, group=4, d=128,
             page=64, len_lo=4001, len_hi=8192, new_lo=2048, new_hi=2048, window=0),
        # small heads without sharing, short odd prompts, small pages and a window
        dict(name="attn_window", op="attn", fmt="e4m3", dtype="bf16", order="hsd", batch=12, heads=12, group=1, d=64,
             page=16, len_lo=77, len_hi=2300, new_lo=33, new_hi=500, window=256),
        # the next token of one sequence
        dict(name="sample_one", op="sample", dtype="fp32", rows=1, vocab=151936, mode="all"),
        # a served batch with mixed settings, logits in bf16 with many ties, an odd vocabulary
        dict(name="sample_batch", op="sample", dtype="bf16", rows=64, vocab=50257, mode="mixed"),
        # every position of a calibration batch sampled at once
        dict(name="sample_rows", op="sample", dtype="fp32", rows=512, vocab=151936, mode="all"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "sample", "sample"])
    if op == "sample":
        return dict(op=op, dtype=rng.choice(["fp32", "bf16", "fp16"]), rows=_log_int(rng, 1, 512),
                    vocab=_log_int(rng, 1000, 151936), mode=rng.choice(["all", "mixed", "topk", "topp", "minp", "free", "greedy"]))
    c = dict(op=op, fmt=rng.choice(["int8", "e4m3"]), order=rng.choice(["hsd", "shd"]), batch=_log_int(rng, 1, 64),
             heads=rng.choice([1, 2, 4, 5, 8, 12]), d=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]))
    hi = _log_int(rng, 1, 32768)
    if op == "attn":
        c["dtype"] = rng.choice(["bf16", "fp16"])
        c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c["window"] = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 2048)
    else:
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        new = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4096) if op == "write" else hi
    hi = max(hi, new)
    c.update(len_hi=hi, len_lo=max(1, hi // rng.choice([1, 2, 8])), new_hi=new, new_lo=max(1, new // rng.choice([1, 3])))
    most = {k: max(work(x)[k] for x in listed() if x["op"] == op) for k in ("bytes", "flops")}
    cells = max(x["batch"] * x["heads"] * x["group"] * x["new_hi"] * x["len_hi"] for x in listed() if x["op"] == "attn")
    while any(work(c)[k] > most[k] for k in most) or (
            op == "attn" and c["batch"] * c["heads"] * c["group"] * c["new_hi"] * c["len_hi"] > cells):
        if c["batch"] > 1:
            c["batch"] -= (c["batch"] + 1) // 2
        else:
            for k in ("len_hi", "len_lo", "new_hi", "new_lo"):
                c[k] = max(1, c[k] // 2)
    return c


def _lengths(case):
    """Tokens of each sequence in the cache after this step, and how many of them are this step's."""
    r = random.Random(1000003 * case["batch"] + case["len_hi"])
    lens = [case["len_hi"]] + [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"] - 1)]
    if case["op"] == "read" or case["new_hi"] == case["len_hi"]:
        return lens, list(lens)
    new = [case["new_hi"]] + [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"] - 1)]
    return lens, [min(a, n) for a, n in zip(lens, new)]


def _visible(case):
    """(query row, cached token) pairs that the causal mask and the window leave."""
    total = 0
    for n, m in zip(*_lengths(case)):
        if case["window"] > 0:
            w = case["window"]
            full = max(0, min(m, n - max(w, n - m)))          # rows that see a whole window
            rest = m - full
            first = n - m + 1
            total += full * w + rest * first + rest * (rest - 1) // 2
        else:
            total += m * (n - m) + m * (m + 1) // 2
    return total


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * SIZE[case["dtype"]] + case["rows"] * 28, "flops": 2 * n}
    lens, new = _lengths(case)
    H, d, page = case["heads"], case["d"], case["page"]
    pages = sum(-(-n // page) - (n - m) // page for n, m in zip(lens, new))
    small = 4 * (2 * len(lens) + 1 + sum(-(-n // page) for n in lens))
    if case["op"] in ("write", "read"):
        rows = sum(new) * H * d
        return {"bytes": 2 * rows * (SIZE[case["dtype"]] + 1) + 8 * pages * H + small, "flops": 4 * rows}
    w = case["window"]
    held = sum(min(n, m + w - 1) if w > 0 else n for n, m in zip(lens, new))
    hq = H * case["group"]
    return {"bytes": 2 * held * H * d + 8 * H * (held // page + len(lens)) + small
            + sum(new) * hq * (2 * d * SIZE[case["dtype"]] + 4),
            "flops": 4 * d * hq * _visible(case)}


# ---------------------------------------------------------------- inputs

def _encode(x, s, fmt):
    """Codes of x at scale s, as bytes; 32 bits throughout."""
    y = torch.where(s > 0, x / s, torch.zeros_like(x))
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _typed(codes, fmt):
    """The cache's bytes as the values they stand for."""
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    if case["op"] == "sample":
        rows, V = case["rows"], case["vocab"]
        logits = randn(rows, V) * 2.5
        top = torch.randint(0, V, (rows, 20), generator=g, device=DEV)
        logits.scatter_add_(1, top, 8 * rand(rows, 20))         # a few likely tokens, as a language model has
        st = dict(case=case, logits=logits.to(TYPES[case["dtype"]]), u=rand(rows))
        mode, one = case["mode"], torch.ones(rows, device=DEV)
        pick = torch.randint(0, 5, (rows,), generator=g, device=DEV)
        temp = 0.6 + 0.6 * rand(rows)
        if mode == "greedy":
            temp = 0 * one
        elif mode == "mixed":
            temp = torch.where(pick == 0, 0 * one, temp)
        st["temperature"] = temp
        k = torch.randint(20, 65, (rows,), generator=g, device=DEV, dtype=torch.int32)
        p, m = 0.85 + 0.13 * rand(rows), 0.02 + 0.08 * rand(rows)
        st["top_k"] = k if mode in ("all", "topk") else torch.where(pick == 1, k, 0 * k) if mode == "mixed" else None
        st["top_p"] = p if mode in ("all", "topp") else torch.where(pick == 2, p, one) if mode == "mixed" else None
        st["min_p"] = m * 0.1 if mode == "all" else m if mode == "minp" else \
            torch.where(pick == 3, m, 0 * one) if mode == "mixed" else None
        return st

    lens, new = _lengths(case)
    B, H, d, page, fmt = case["batch"], case["heads"], case["d"], case["page"], case["fmt"]
    held = [-(-n // page) for n in lens]
    pages, width = sum(held) + 3, max(held)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    ids, at = order.cpu(), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new, dtype=torch.int32).cumsum(0)
    st = dict(case=case, table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu=cu.to(DEV),
              rows=sum(new))
    for name in ("k", "v"):
        shape = (pages, H, page, d) if case["order"] == "hsd" else (pages, page, H, d)
        codes = torch.empty(shape, dtype=torch.uint8, device=DEV)
        if case["order"] == "shd":
            codes = codes.permute(0, 2, 1, 3)
        scales = torch.empty(pages, H, device=DEV)
        step = max(1, (1 << 27) // (H * page * d))
        loud = 1 + 5 * (rand(d) < 0.03).float() if name == "k" else torch.ones(d, device=DEV)   # channels that keys raise
        for i in range(0, pages, step):
            x = randn(min(step, pages - i), H, page, d) * loud
            s = x.abs().amax((2, 3)) / QMAX[fmt]
            codes[i:i + step] = _encode(x, s[:, :, None, None], fmt)
            scales[i:i + step] = s
        st[name + "_codes"], st[name + "_scales"] = codes, scales
    t = TYPES[case["dtype"]]
    if case["op"] == "write":
        st["k"], st["v"] = randn(sum(new), H, d).to(t), randn(sum(new), H, d).to(t)
    if case["op"] == "attn":
        st["q"] = (1.5 * randn(sum(new), H * case["group"], d)).to(t)
    return st


# ---------------------------------------------------------------- plain forms

def _rows(st):
    """Sequence and position of every row."""
    t = torch.arange(st["rows"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(st["cu"], t, right=True) - 1
    pos = st["lens"][b].long() - st["cu"][b + 1].long() + t.long()
    return b, pos


def _plain_write(st):
    c = st["case"]
    page, fmt = c["page"], c["fmt"]
    b, pos = _rows(st)
    pid, slot = st["table"][b, pos // page].long(), pos % page
    pos0 = st["lens"].long() - (st["cu"][1:] - st["cu"][:-1]).long()
    first = st["table"][torch.arange(c["batch"], device=DEV), (pos0 // page)].long()
    lo = pos0 % page                                            # old tokens in each sequence's first page
    out = {}
    for name in ("k", "v"):
        codes, scales = st[name + "_codes"], st[name + "_scales"]
        x = torch.nan_to_num(st[name].float(), nan=0.0)
        amax = torch.zeros_like(scales).index_reduce_(0, pid, x.abs().amax(2), "amax")
        s = amax / QMAX[fmt]
        old = scales[first]
        s[first] = torch.where(lo[:, None] > 0, torch.maximum(old, s[first]), s[first])
        # old codes of a page that a louder row has joined move to the new scale
        part = codes[first]
        moved = _encode(_decode(part, fmt) * old[:, :, None, None], s[first][:, :, None, None], fmt)
        keep = (torch.arange(page, device=DEV)[None, None, :, None] < lo[:, None, None, None]) & \
            (s[first] > old)[:, :, None, None]
        codes[first] = torch.where(keep, moved, part)
        codes[pid, :, slot] = _encode(x, s[pid][:, :, None], fmt)
        scales[pid] = s[pid]
        out[name + "_codes"], out[name + "_scales"] = _typed(codes, fmt), scales
    return out


def _plain_read(st):
    c = st["case"]
    b, pos = _rows(st)
    pid, slot = st["table"][b, pos // c["page"]].long(), pos % c["page"]
    return {name: (_decode(st[name + "_codes"][pid, :, slot], c["fmt"]) * st[name + "_scales"][pid][:, :, None])
            .to(TYPES[c["dtype"]]) for name in ("k", "v")}


def _plain_attn(st):
    c = st["case"]
    B, H, G, d, page = c["batch"], c["heads"], c["group"], c["d"], c["page"]
    n_new = (st["cu"][1:] - st["cu"][:-1]).long()
    lens = st["lens"].long()
    Q = c["new_hi"]
    i = torch.arange(Q, device=DEV)
    at = (st["cu"][:-1].long()[:, None] + i).clamp(max=st["rows"] - 1)
    q = st["q"][at].float().view(B, Q, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, d)
    table = st["table"].long().clamp(min=0)
    L = table.shape[1] * page
    j = torch.arange(L, device=DEV)

    def held(name):
        x = _decode(st[name + "_codes"][table], c["fmt"]) * st[name + "_scales"][table][:, :, :, None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, d)

    s = torch.matmul(q, held("k").transpose(2, 3).contiguous()) * (1.0 / math.sqrt(d))
    pos = (lens - n_new)[:, None] + i                                                   # [B, Q]
    seen = (j <= pos[:, :, None]) & (j < lens[:, None, None])
    if c["window"] > 0:
        seen &= j > pos[:, :, None] - c["window"]
    s = s.view(B, H, G, Q, L).masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(4, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = s.sub_(m).exp_()
    z = p.sum(4, keepdim=True)
    o = torch.matmul(p.view(B, H, G * Q, L), held("v")).view(B, H, G, Q, d)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    lse = (m + z.log())[..., 0]
    b, posr = _rows(st)
    r = posr - (lens - n_new)[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, r].reshape(st["rows"], H * G, d).to(st["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2)[b, r].reshape(st["rows"], H * G)}


def _plain_sample(st):
    l = st["logits"].float()
    rows, V = l.shape
    l = torch.nan_to_num(l, nan=float("-inf"), posinf=torch.finfo(torch.float32).max, neginf=float("-inf"))
    T = st["temperature"].double()[:, None]
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    w = ((val.double() - val[:, :1].double()) / T).exp()
    rank = torch.arange(V, device=DEV)
    keep = torch.ones_like(w, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        keep &= (rank < k) | (k <= 0)
    wk = torch.where(keep, w, torch.zeros_like(w))
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        before = wk.cumsum(1) - wk
        keep &= (before < p * wk.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
    if st["min_p"] is not None:
        keep &= w >= st["min_p"].double()[:, None].clamp(max=1)
    wi = torch.zeros_like(w).scatter_(1, idx, torch.where(keep, w, torch.zeros_like(w)))
    cum = wi.cumsum(1)
    total = cum[:, -1:]
    token = (cum <= st["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    logprob = (wi.gather(1, token) / total).log()
    greedy = T <= 0
    token = torch.where(greedy, idx[:, :1], token)
    logprob = torch.where(greedy, torch.zeros_like(logprob), logprob)
    return {"tokens": token[:, 0].to(torch.int32), "logprobs": logprob[:, 0].float()}


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import weight_only_mixed_amd as slq
    c = st["case"]
    if c["op"] == "sample":
        tokens, logprobs = slq.slq_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                          top_p=st["top_p"], min_p=st["min_p"])
        return {"tokens": tokens, "logprobs": logprobs}
    fmt = slq.SLQ_KV_INT8 if c["fmt"] == "int8" else slq.SLQ_KV_E4M3
    cache = slq.KvCache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], fmt)
    seqs = slq.KvSeqs(st["table"], st["lens"], st["cu"])
    if c["op"] == "write":
        slq.slq_kv_write(cache, seqs, st["k"], st["v"], max_new=c["new_hi"])
        return {"k_codes": _typed(st["k_codes"], c["fmt"]), "k_scales": st["k_scales"],
                "v_codes": _typed(st["v_codes"], c["fmt"]), "v_scales": st["v_scales"]}
    if c["op"] == "read":
        k, v = slq.slq_kv_read(cache, seqs, st["rows"], TYPES[c["dtype"]], max_rows=c["len_hi"])
        return {"k": k, "v": v}
    out, lse = slq.slq_kv_attention(cache, seqs, st["q"], window=c["window"], max_q=c["new_hi"], max_len=c["len_hi"],
                                    with_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn,
            "sample": _plain_sample}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits

def _value64(codes, fmt):
    """Bytes as numbers, from the formats' definitions."""
    u = codes.to(torch.int64)
    if fmt == "int8":
        return torch.where(u > 127, u - 256, u).double()
    sign = 1.0 - 2.0 * (u >> 7).double()
    e, m = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.pow(2.0, (e - 10).double()))
    return sign * v


def _nearest64(y, fmt):
    """The nearest value that a code stands for, ties to even."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    y = y.clamp(-448, 448)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(2.0, e - 3)
    return torch.round(y / step) * step


def _exact_write(case, st):
    page, fmt = case["page"], case["fmt"]
    out = {}
    lens, new = _lengths(case)
    table, cu = st["table"].cpu(), st["cu"].cpu()
    for name in ("k", "v"):
        val = _value64(st[name + "_codes"], fmt) if fmt == "e4m3" else None
        scales = st[name + "_scales"].double()
        for b, (n, m) in enumerate(zip(lens, new)):
            x = st[name][int(cu[b]):int(cu[b + 1])].double()
            for pg in range((n - m) // page, -(-n // page)):
                lo, hi = max(0, n - m - pg * page), min(page, n - pg * page)
                rows = x[pg * page + lo - (n - m):pg * page + hi - (n - m)]
                p = int(table[b, pg])
                s = rows.abs().amax((0, 2)) / QMAX[fmt]
                if lo > 0:
                    s = torch.maximum(s, scales[p])
                if val is not None:
                    if lo > 0:
                        moved = _nearest64(val[p, :, :lo] * (scales[p] / s)[:, None, None], fmt)
                        val[p, :, :lo] = torch.where((s > scales[p])[:, None, None], moved, val[p, :, :lo])
                    val[p, :, lo:hi] = _nearest64(rows.permute(1, 0, 2) / s[:, None, None], fmt)
                scales[p] = s
        out[name + "_codes"], out[name + "_scales"] = val, scales
    return out


def _exact_rows(case, st, name, b, n):
    """The first n tokens of sequence b: [heads, n, d] in 64 bits."""
    ids = st["table"][b, :-(-n // case["page"])].long()
    x = _value64(st[name + "_codes"][ids], case["fmt"]) * st[name + "_scales"][ids].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(case["heads"], -1, case["d"])[:, :n]


def _exact_attn(case, st):
    H, G, d = case["heads"], case["group"], case["d"]
    outs, lses, at = [], [], 0
    for b, (n, m) in enumerate(zip(*_lengths(case))):
        first = max(0, n - m - case["window"] + 1) if case["window"] > 0 else 0
        K, V = _exact_rows(case, st, "k", b, n)[:, first:], _exact_rows(case, st, "v", b, n)[:, first:]
        q = st["q"][at:at + m].double().view(m, H, G, d)
        pos = torch.arange(n - m, n, device=DEV)[:, None]
        j = torch.arange(first, n, device=DEV)[None]
        hide = (j > pos) | (j <= pos - case["window"] if case["window"] > 0 else j < 0)
        o = torch.empty(m, H, G, d, dtype=torch.float64, device=DEV)
        lse = torch.empty(m, H, G, dtype=torch.float64, device=DEV)
        for h in range(H):
            s = (q[:, h].reshape(m * G, d) @ K[h].t().contiguous() / math.sqrt(d)).view(m, G, -1)
            s.masked_fill_(hide[:, None], float("-inf"))
            lse[:, h] = torch.logsumexp(s, 2)
            o[:, h] = (torch.softmax(s, 2).view(m * G, -1) @ V[h]).view(m, G, d)
        outs.append(o.view(m, H * G, d))
        lses.append(lse.view(m, H * G))
        at += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_sample(case, st):
    tokens, logprobs = [], []
    for r in range(case["rows"]):
        l = st["logits"][r].double()
        T = float(st["temperature"][r])
        if T <= 0:
            tokens.append(int((l == l.max()).nonzero()[0, 0]))
            logprobs.append(0.0)
            continue
        w = torch.exp((l - l.max()) / T)
        order = torch.argsort(-l, stable=True)
        n = len(l)
        if st["top_k"] is not None and int(st["top_k"][r]) > 0:
            n = min(n, int(st["top_k"][r]))
        ws = w[order]
        cut = n
        if st["top_p"] is not None and float(st["top_p"][r]) < 1:
            reach = torch.cumsum(ws[:n], 0) >= float(st["top_p"][r]) * ws[:n].sum()
            cut = min(cut, int(reach.nonzero()[0, 0]) + 1 if bool(reach.any()) else n)
        if st["min_p"] is not None:
            cut = min(cut, int((ws >= min(1.0, float(st["min_p"][r]))).sum()))
        kept = order[:cut].sort().values
        cum = torch.cumsum(w[kept], 0)
        i = min(int((cum <= float(st["u"][r]) * cum[-1]).sum()), cut - 1)
        tokens.append(int(kept[i]))
        logprobs.append(float(torch.log(w[kept[i]] / cum[-1])))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "logprobs": torch.tensor(logprobs, dtype=torch.float64)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, st)
    if case["op"] == "read":
        lens, _ = _lengths(case)
        return {name: torch.cat([_exact_rows(case, st, name, b, n).permute(1, 0, 2) for b, n in enumerate(lens)])
                for name in ("k", "v")}
    return _exact_attn(case, st) if case["op"] == "attn" else _exact_sample(case, st)
