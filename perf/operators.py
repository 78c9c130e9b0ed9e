"""Cases of the decode-step operators around the quantized projections: page tables built
on the device, the paged key-value cache and its attention, and the RMS norm that feeds the
projections.

`run` computes a case's operator in its plain form (elementary torch operations in float32,
integers in int64), or, with `own` true, through gemv_prefill_decode_amd.

A case's "op" is one of

  extend  block tables, sequence lengths, slots and positions of a step's new tokens
  append  new keys and values written into their slots of the paged cache
  attend  attention of one new token per sequence over the paged cache
  norm    residual addition and RMS norm, to float32 or to Q8_1 codes with scales

The cache holds pages of `page` tokens, [n_pages, n_kv, page, head_dim] (layout "hnd") or
[n_pages, page, n_kv, head_dim] ("nhd"), as float16, bfloat16 or 8-bit codes ("q8": int8
and one float32 scale per token and head).
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "q8": torch.int8}


def _row_bytes(case):
    """Bytes of one token's key (or value) of one head in the cache: its elements, and a q8 row's scale."""
    return case["head_dim"] + 4.0 if case["kind"] == "q8" else 2.0 * case["head_dim"]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a full serving batch: one new token per sequence
        dict(name="extend_decode_64", op="extend", batch=64, max_len=4096, max_new=1, page=16, pad=0, short=0),
        # admission of many prompts at once, their rows padded to a bucket
        dict(name="extend_prompts_512", op="extend", batch=512, max_len=2048, max_new=512, page=32, pad=1000, short=0),
        # the LFM2.5-350M-shaped decode step (8 heads of 64, 16 query heads) of a small batch
        dict(name="append_decode_16", op="append", tokens=16, run=1, n_kv=8, group=2, head_dim=64, page=16,
             kind="f16", layout="hnd", pad=0),
        # a chunk of prompts written at once, heads of 128 as in an 8B-class model
        dict(name="append_prompts_8192", op="append", tokens=8192, run=1024, n_kv=8, group=4, head_dim=128,
             page=32, kind="bf16", layout="nhd", pad=64),
        # one user, a short context: the latency of a single call
        dict(name="attend_one_short", op="attend", batch=1, max_len=97, n_kv=8, group=2, head_dim=64, page=16,
             kind="f16", layout="hnd", even=1, pad=0),
        # one user, a very long context: the work has to be split along the cache
        dict(name="attend_one_long", op="attend", batch=1, max_len=131071, n_kv=8, group=4, head_dim=128, page=64,
             kind="f16", layout="hnd", even=1, pad=0),
        # a serving batch of mixed lengths, padded to a captured batch size
        dict(name="attend_batch_ragged", op="attend", batch=48, max_len=16384, n_kv=8, group=4, head_dim=128,
             page=16, kind="bf16", layout="nhd", even=0, pad=3),
        # a large batch on the 8-bit cache
        dict(name="attend_batch_q8", op="attend", batch=64, max_len=8192, n_kv=8, group=8, head_dim=128, page=32,
             kind="q8", layout="hnd", even=0, pad=0),
        # the norm before a single token's projections
        dict(name="norm_one", op="norm", rows=1, k=1024, out="f32", residual=1),
        # the norm before a decode batch's MoE gate/up on Q8_1 activations
        dict(name="norm_q8_16", op="norm", rows=16, k=4096, out="q8", residual=1),
        # the norm of a 2048-token prefill, 8B-class width
        dict(name="norm_prefill_2048", op="norm", rows=2048, k=4096, out="f32", residual=1),
        # a prefill's norm to Q8_1, one of the rarer widths
        dict(name="norm_q8_1000", op="norm", rows=1000, k=4608, out="q8", residual=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "append", "attend", "attend", "norm"])
    if op == "extend":
        return dict(op=op, batch=_log_int(rng, 1, 1024), max_len=_log_int(rng, 1, 16384),
                    max_new=_log_int(rng, 1, 512), page=rng.choice([1, 8, 16, 32, 64, 128]), pad=rng.randint(0, 300),
                    short=rng.randint(0, 1))
    if op == "append":
        n_kv, head_dim = rng.choice([1, 2, 3, 4, 8, 16]), 32 * rng.randint(1, 8)
        most = max(1, 8192 * 8 * 128 // (n_kv * head_dim))
        return dict(op=op, tokens=_log_int(rng, 1, min(8192, most)), run=_log_int(rng, 1, 1024), n_kv=n_kv,
                    group=rng.randint(1, 8), head_dim=head_dim, page=rng.choice([1, 8, 16, 32, 64, 128]),
                    kind=rng.choice(["f16", "bf16", "q8"]), layout=rng.choice(["hnd", "nhd"]), pad=rng.randint(0, 9))
    if op == "attend":
        n_kv, head_dim, batch = rng.choice([1, 2, 3, 4, 8, 16]), 32 * rng.randint(1, 8), _log_int(rng, 1, 64)
        most = max(1, 48 * 8192 * 8 * 128 // (n_kv * head_dim * batch))
        return dict(op=op, batch=batch, max_len=_log_int(rng, 1, min(65536, most)), n_kv=n_kv,
                    group=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 20]), head_dim=head_dim,
                    page=rng.choice([1, 8, 16, 32, 64, 128]), kind=rng.choice(["f16", "bf16", "q8"]),
                    layout=rng.choice(["hnd", "nhd"]), even=rng.randint(0, 1), pad=rng.randint(0, 3))
    k = 32 * _log_int(rng, 1, 512)
    return dict(op=op, rows=_log_int(rng, 1, max(1, min(4096, 2048 * 4096 // k))), k=k, out=rng.choice(["f32", "q8"]),
                residual=rng.randint(0, 1))


def _spread(n, most, least=1):
    """n lengths up to `most`, quadratically spread: few long ones, many short ones."""
    return [max(least, int(round(most * ((i + 1) / n) ** 2))) for i in range(n)]


def _lens(case):
    full = [case["max_len"]] * case["batch"] if case["even"] else _spread(case["batch"], case["max_len"])
    return full + [0] * case["pad"]


def _new_lens(case):
    return [1] * case["batch"] if case["max_new"] == 1 else _spread(case["batch"], case["max_new"], 0)


def work(case):
    if case["op"] == "extend":
        b, rows = case["batch"], sum(_new_lens(case)) + case["pad"]
        return {"bytes": 12.0 * b + 8.0 * sum(_new_lens(case)) / case["page"] + 8.0 * rows + 4, "flops": 0.0}
    if case["op"] == "append":
        n = case["tokens"] * case["n_kv"]
        return {"bytes": 2 * n * (4.0 * case["head_dim"] + _row_bytes(case)) + 4.0 * (case["tokens"] + case["pad"]), "flops": 0.0}
    if case["op"] == "attend":
        lens, hq = _lens(case), case["n_kv"] * case["group"]
        kv = sum(lens) * case["n_kv"]
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * kv * _row_bytes(case) + len(lens) * (8.0 * hq * case["head_dim"] + 4 * hq + 4) + 4.0 * pages,
                "flops": 4.0 * kv * case["group"] * case["head_dim"]}
    n = case["rows"] * case["k"]
    return {"bytes": n * (4 + (1.125 if case["out"] == "q8" else 4) + (8 if case["residual"] else 0)) + 4.0 * case["k"],
            "flops": 5.0 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(g, case, n_pages, filled):
    """An empty (or filled) cache: k, v as [n_pages, n_kv, page, head_dim] views, and the 8-bit scales."""
    hnd = case["layout"] == "hnd"
    shape = [n_pages, case["n_kv"], case["page"]] if hnd else [n_pages, case["page"], case["n_kv"]]
    d, out = case["head_dim"], []
    for _ in range(2):
        t = torch.zeros(shape + [d], dtype=DTYPES[case["kind"]], device="cuda")
        s = torch.zeros(shape, device="cuda") if case["kind"] == "q8" else None
        if filled:
            step = max(1, (1 << 25) // max(1, t[0].numel()))
            for i in range(0, n_pages, step):
                part = _randn(g, *t[i:i + step].shape)
                t[i:i + step] = (part * 42).round_().clamp_(-127, 127) if s is not None else part
            if s is not None:
                s.copy_((torch.rand(s.shape, generator=g, device="cuda") + 0.5) * (3.0 / 127))
        out.append((t if hnd else t.transpose(1, 2), s if s is None or hnd else s.transpose(1, 2)))
    (k, ks), (v, vs) = out
    return {"k": k, "v": v, "ks": ks, "vs": vs}


def _handle(cache):
    import gemv_prefill_decode_amd as qmm

    return qmm.KVCache(cache["k"], cache["v"], cache["ks"], cache["vs"])


def prepare(case, seed):
    g = _gen(seed)
    state = {"case": case, "seed": seed}
    if case["op"] == "extend":
        b, ps = case["batch"], case["page"]
        cached = torch.tensor(_spread(b, case["max_len"], 0), device="cuda")[_perm(g, b)]
        new = torch.tensor(_new_lens(case), device="cuda")[_perm(g, b)]
        have, total = (cached + ps - 1) // ps, (cached + new + ps - 1) // ps
        width = -(-(case["max_len"] + case["max_new"]) // ps)
        ids = _perm(g, int(total.sum()) + 64)
        col = torch.arange(width, device="cuda")
        at = (have.cumsum(0) - have)[:, None] + col
        table = torch.where(col < have[:, None], ids[at.clamp(max=ids.numel() - 1)], -1)
        free = ids[int(have.sum()):]
        if case["short"]:  # the free list runs dry for the last sequences
            free = free[: int((total - have).sum()) * 3 // 4]
        n_rows = sum(_new_lens(case)) + case["pad"]
        out = {"seq_lens": torch.empty(b, dtype=torch.int32, device="cuda"), "pages_used": torch.empty(1, dtype=torch.int32, device="cuda")}
        out |= {n: torch.empty(n_rows, dtype=torch.int32, device="cuda") for n in ("slots", "positions")}
        state |= {"table": table.int().contiguous(), "cached": cached.int(), "new": new.int(),
                  "free": free.int().contiguous(), "n_rows": n_rows, "out": out}
    elif case["op"] == "append":
        n, ps, run_ = case["tokens"], case["page"], min(case["run"], case["tokens"])
        seqs, per = -(-n // run_), -(-run_ // ps)
        cache = _pages(g, case, seqs * per + 4, False)
        pages = _perm(g, seqs * per + 4)
        j = torch.arange(n, device="cuda")
        slots = pages[(j // run_) * per + (j % run_) // ps] * ps + (j % run_) % ps
        d, kv = case["head_dim"], case["n_kv"]
        qkv = _randn(g, n + case["pad"], (case["group"] + 2) * kv * d)  # the fused projection's output
        k, v = (qkv[:, i * kv * d:(i + 1) * kv * d].unflatten(1, (kv, d)) for i in (case["group"], case["group"] + 1))
        state |= {"cache": cache, "knew": k, "vnew": v,
                  "slots": torch.cat([slots, slots.new_full((case["pad"],), -1)]).int()}
        if own:
            state["handle"] = _handle(cache)
    elif case["op"] == "attend":
        ps, lens = case["page"], torch.tensor(_lens(case), device="cuda")
        lens = torch.cat([lens[: case["batch"]][_perm(g, case["batch"])], lens[case["batch"]:]])
        pages = (lens + ps - 1) // ps
        n_pages, width = int(pages.sum()) + 4, max(1, -(-case["max_len"] // ps))
        cache = _pages(g, case, n_pages, True)
        ids = _perm(g, n_pages)
        at = (pages.cumsum(0) - pages)[:, None] + torch.arange(width, device="cuda")
        # entries behind a sequence's last page are what an earlier user of the row left
        table = torch.where(torch.arange(width, device="cuda") < pages[:, None], ids[at.clamp(max=n_pages - 1)], -1)
        hq, d = case["n_kv"] * case["group"], case["head_dim"]
        q = 1.5 * _randn(g, lens.numel(), hq, d)
        state |= {"cache": cache, "q": q, "table": table.int().contiguous(), "lens": lens.int(),
                  "out": torch.empty_like(q), "lse": torch.empty(lens.numel(), hq, device="cuda")}
        if own:
            state["handle"] = _handle(cache)
    else:
        n, k = case["rows"], case["k"]
        state |= {"x": _randn(g, n, k), "r": 3 * _randn(g, n, k) if case["residual"] else None,
                  "w": 1 + 0.2 * _randn(g, k)}
        state |= {"h": torch.empty(n, k, device="cuda") if case["residual"] else None,
                  "y": torch.empty(n, k, device="cuda") if case["out"] == "f32" else None}
        if case["out"] == "q8":
            state |= {"q": torch.empty(n, k, dtype=torch.int8, device="cuda"), "d": torch.empty(n, k // 32, device="cuda")}
    return state


# ------------------------------------------------------------------ plain forms
def _q8_values(codes, scales):
    """The values that codes [.., n] and their scales [..] stand for, in one operation."""
    return torch.mul(codes, scales.unsqueeze(-1))


def _q8_codes(z):
    """(codes, scales) of z's last axis: d = max|z|/127, codes z*(1/d) rounded half away from
    zero, each step in float32."""
    top = z.abs().amax(-1, keepdim=True)
    d = top / torch.full_like(top, 127.0)
    d = torch.where(d < 2.0 ** -126, torch.zeros_like(d), d)
    c = z * torch.where(d > 0, torch.ones_like(d) / d, torch.zeros_like(d))
    whole = c.trunc()
    codes = whole + torch.where((c - whole).abs() >= 0.5, c.sign(), torch.zeros_like(c))
    return codes.to(torch.int8), d.squeeze(-1)


def _plain_extend(s):
    ps, table = s["case"]["page"], s["table"]
    cached, new, free = s["cached"].long(), s["new"].long(), s["free"].long()
    width, n_free = table.shape[1], free.numel()
    rows = new.clamp(min=0)
    have = (cached.clamp(min=0) + ps - 1) // ps
    bad = (cached < 0) | (new < 0) | (cached + new > width * ps)
    need = torch.where(bad, 0, (cached + new + ps - 1) // ps - have)
    first = need.cumsum(0) - need
    bad = bad | ((need > 0) & (first + need > n_free))
    col = torch.arange(width, device="cuda")
    take = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None]) & ~bad[:, None]
    if n_free:
        table.copy_(torch.where(fresh, free[take.clamp(0, n_free - 1)].int(), table))
    ends = rows.cumsum(0)
    j = torch.arange(s["n_rows"], device="cuda")
    seq = torch.searchsorted(ends, j, right=True)
    real = seq < cached.numel()
    seq = seq.clamp(max=cached.numel() - 1)
    pos = cached[seq] + j - (ends - rows)[seq]
    page = table[seq, (pos // ps).clamp(0, width - 1)].long()
    slots = torch.where(real & ~bad[seq] & (page >= 0), page * ps + pos % ps, -1)
    return {"table": table, "seq_lens": torch.where(bad, cached, cached + new).int(), "slots": slots.int(),
            "positions": torch.where(real, pos, -1).int(), "pages_used": need.sum().reshape(1).int()}


def _plain_append(s):
    case, c = s["case"], s["cache"]
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    page, at = slots // case["page"], slots % case["page"]
    for new, codes, scales in ((s["knew"], c["k"], c["ks"]), (s["vnew"], c["v"], c["vs"])):
        if scales is None:
            codes[page, :, at] = new[live].to(codes.dtype)
        else:
            codes[page, :, at], scales[page, :, at] = _q8_codes(new[live])
    return _cache_values(c)


def _cache_values(c):
    """The whole cache, 8-bit pages as the values they stand for."""
    if c["ks"] is None:
        return {"k": c["k"], "v": c["v"]}
    return {"k": _q8_values(c["k"], c["ks"]), "v": _q8_values(c["v"], c["vs"])}


def _plain_gather(pages, scales, table):
    """The cache's rows of every sequence in order: float32 [batch, n_kv, width * page, head_dim]."""
    rows = pages[table].transpose(1, 2).flatten(2, 3).float()
    return rows if scales is None else rows * scales[table].transpose(1, 2).flatten(2, 3).unsqueeze(-1)


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    table = s["table"].long().clamp(min=0)
    b, hq, d = s["q"].shape
    q = s["q"].reshape(b, case["n_kv"], case["group"], d)
    dead = torch.arange(table.shape[1] * case["page"], device="cuda") >= s["lens"][:, None]
    score = (q @ _plain_gather(c["k"], c["ks"], table).transpose(-1, -2)) * d ** -0.5
    score = score.masked_fill(dead[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    v = _plain_gather(c["v"], c["vs"], table).masked_fill(dead[:, None, :, None], 0.0)
    out = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    return {"out": out.reshape(b, hq, d), "lse": (top + torch.log(total)).reshape(b, hq)}


def _plain_norm(s):
    h = s["x"] if s["r"] is None else s["x"] + s["r"]
    inv = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    more = {} if s["r"] is None else {"h": h}
    if s["case"]["out"] == "f32":
        return {"y": h * inv * s["w"], **more}
    # 1/rms is one factor of a whole row: the codes are those of h*w, the scales carry it
    q, d = _q8_codes((h * s["w"]).unflatten(-1, (-1, 32)))
    return {"y": _q8_values(q, d * inv), **more}


PLAIN = {"extend": _plain_extend, "append": _plain_append, "attend": _plain_attend, "norm": _plain_norm}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import gemv_prefill_decode_amd as qmm

    op = s["case"]["op"]
    if op == "extend":
        qmm.paged_extend(s["table"], s["cached"], s["new"], s["free"], s["case"]["page"], s["n_rows"], **s["out"])
        return {"table": s["table"], **s["out"]}
    if op == "append":
        qmm.kv_append(s["handle"], s["knew"], s["vnew"], s["slots"])
        return _cache_values(s["cache"])
    if op == "attend":
        qmm.paged_attention(s["q"], s["handle"], s["table"], s["lens"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    more = {} if s["r"] is None else {"h": s["h"]}
    if s["case"]["out"] == "f32":
        qmm.add_rmsnorm(s["x"], s["w"], s["r"], eps=EPS, y=s["y"], h=s["h"])
        return {"y": s["y"], **more}
    qmm.add_rmsnorm_q8(s["x"], s["w"], s["r"], eps=EPS, q=s["q"], d=s["d"], h=s["h"])
    return {"y": _q8_values(s["q"].unflatten(-1, (-1, 32)), s["d"]), **more}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_codes(z, n):
    """Codes (float64) and scales of float32 values in runs of n: the rule that decides integer
    codes is itself in float32."""
    import numpy as np

    z = np.asarray(z, dtype=np.float32).reshape(-1, n)
    d = np.abs(z).max(axis=1) / np.float32(127)
    d[d < np.float32(2.0 ** -126)] = 0
    inv = np.divide(np.float32(1), d, out=np.zeros_like(d), where=d > 0)
    c = (z * inv[:, None]).astype(np.float64)
    return np.sign(c) * np.floor(np.abs(c) + 0.5), d.astype(np.float64)


def _exact_extend(s):
    ps, table = s["case"]["page"], s["table"].tolist()
    cached, new, free = s["cached"].tolist(), s["new"].tolist(), s["free"].tolist()
    used, lens, slots, positions = 0, [], [], []
    for row, c, n in zip(table, cached, new):
        have = -(-c // ps)
        need = -(-(c + n) // ps) - have if c + n <= len(row) * ps else 0
        ok = c + n <= len(row) * ps and (need == 0 or used + need <= len(free))
        if ok:
            row[have:have + need] = free[used:used + need]
        used += need
        lens.append(c + n if ok else c)
        positions += range(c, c + n)
        slots += [row[p // ps] * ps + p % ps if ok and row[p // ps] >= 0 else -1 for p in range(c, c + n)]
    rest = [-1] * (s["n_rows"] - len(slots))
    return {"table": _ints(table), "seq_lens": _ints(lens), "slots": _ints(slots + rest),
            "positions": _ints(positions + rest), "pages_used": _ints([used])}


def _exact_append(s):
    case, slots, out = s["case"], s["slots"].cpu().numpy(), {}
    for name, new in (("k", s["knew"]), ("v", s["vnew"])):
        whole = s["cache"][name].double() if case["kind"] != "q8" else torch.zeros(s["cache"][name].shape, dtype=torch.float64, device="cuda")
        rows = new.contiguous()
        if case["kind"] == "q8":
            codes, scales = _exact_codes(rows.cpu().numpy(), case["head_dim"])
            rows = torch.from_numpy((codes * scales[:, None]).reshape(rows.shape)).to("cuda")
        live = torch.from_numpy((slots >= 0).nonzero()[0]).to("cuda")
        at = s["slots"].long()[live]
        whole[at // case["page"], :, at % case["page"]] = rows.double()[live]
        out[name] = whole
    return out


def _exact_attend(s):
    case, c, ps = s["case"], s["cache"], s["case"]["page"]
    b, hq, d = s["q"].shape
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        page, at = s["table"][i].long()[t // ps], t % ps
        for h in range(case["n_kv"]):
            kv = []
            for x, sc in ((c["k"], c["ks"]), (c["v"], c["vs"])):
                x = x[page, h, at].double()
                kv.append(x if sc is None else x * sc[page, h, at].double()[:, None])
            mine = slice(h * case["group"], (h + 1) * case["group"])
            score = torch.mv(kv[0], s["q"][i, mine].double()[0])[None] if case["group"] == 1 else s["q"][i, mine].double() @ kv[0].T.contiguous()
            score = score / math.sqrt(d)
            lse[i, mine] = torch.logsumexp(score, -1)
            out[i, mine] = torch.exp(score - lse[i, mine][:, None]) @ kv[1]
    return {"out": out, "lse": lse}


def _exact_norm(s):
    h32 = s["x"] if s["r"] is None else s["x"] + s["r"]
    h, w = h32.double(), s["w"].double()
    rms = torch.sqrt(h.pow(2).sum(-1, keepdim=True) / h.shape[1] + EPS)
    more = {} if s["r"] is None else {"h": s["x"].double() + s["r"].double()}
    if s["case"]["out"] == "f32":
        return {"y": h / rms * w, **more}
    codes, scales = _exact_codes((h32 * s["w"]).cpu().numpy(), 32)
    y = torch.from_numpy(codes * scales[:, None]).to("cuda").reshape(h.shape[0], -1, 32)
    return {"y": y / rms.unsqueeze(-1), **more}


EXACT = {"extend": _exact_extend, "append": _exact_append, "attend": _exact_attend, "norm": _exact_norm}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
