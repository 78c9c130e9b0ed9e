"""Cases of the operators on microscaled 4-bit floats (MXFP4: E2M1 codes, one E8M0 scale per 32
values): quantization of activations and weights, the RMS norm that writes them, the product of two
MXFP4 matrices, and the paged key-value cache in this format with its append and attention.

`run` computes a case's operator in its plain form (elementary torch operations in float32,
integers in int32 or int64), or, with `own` true, through gemv_prefill_decode_amd.

A case's "op" is one of

  quant   rows to codes and scales, and back to the values they stand for
  norm    residual addition and RMS norm, the result in MXFP4 with one float32 factor per row
  gemm    dst[n, m] = x[n, k] w[m, k]^T, both in MXFP4, with or without a factor per row of x
  append  new keys and values written into their slots of the paged MXFP4 cache
  attend  attention of one new token per sequence over it

Codes are uint8 [.., k/2], element 2j in the low nibble of byte j; scales uint8 [.., k/32], 2^(byte - 127).
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MX_BYTES = 0.5 + 1.0 / 32      # of one element


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's activations before a projection of the LFM2.5-350M shape
        dict(name="quant_one", op="quant", rows=1, k=1024, type="f32"),
        # the activations of a 2048-token prefill before an 8B-class down projection
        dict(name="quant_prefill_2048", op="quant", rows=2048, k=14336, type="f32"),
        # the norm of a decode batch before its projections
        dict(name="norm_16", op="norm", rows=16, k=4096, residual=1),
        # the norm of a 2048-token prefill
        dict(name="norm_prefill_2048", op="norm", rows=2048, k=4096, residual=1),
        # one token through the LFM2.5-350M feed-forward gate: latency
        dict(name="gemm_one", op="gemm", m=4608, k=1024, n=1, scaled=1),
        # a decode batch through an 8B-class gate: the weights' bytes
        dict(name="gemm_decode_16", op="gemm", m=14336, k=4096, n=16, scaled=1),
        # a 512-token prefill through the LFM2.5-350M down projection: few tiles, a long sum
        dict(name="gemm_down_512", op="gemm", m=1024, k=4608, n=512, scaled=0),
        # a 2048-token prefill through an 8B-class gate: the matrix cores
        dict(name="gemm_prefill_2048", op="gemm", m=14336, k=4096, n=2048, scaled=1),
        # the LFM2.5-350M-shaped decode step of a small batch
        dict(name="append_decode_16", op="append", tokens=16, run=1, n_kv=8, group=2, head_dim=64, page=16,
             layout="hnd", pad=0),
        # a chunk of prompts written at once, heads of 128 as in an 8B-class model
        dict(name="append_prompts_8192", op="append", tokens=8192, run=1024, n_kv=8, group=4, head_dim=128, page=32,
             layout="nhd", pad=64),
        # one user, a very long context: the work has to be split along the cache
        dict(name="attend_one_long", op="attend", batch=1, max_len=131071, n_kv=8, group=4, head_dim=128, page=64,
             layout="hnd", even=1, pad=0),
        # a serving batch of mixed lengths, padded to a captured batch size
        dict(name="attend_batch_ragged", op="attend", batch=61, max_len=16384, n_kv=8, group=8, head_dim=128, page=16,
             layout="nhd", even=0, pad=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "norm", "gemm", "gemm", "append", "attend", "attend"])
    if op in ("quant", "norm"):
        k = 32 * _log_int(rng, 1, 512)
        rows = _log_int(rng, 1, max(1, min(8192, (2048 * 14336 if op == "quant" else 2048 * 4096) // k)))
        if op == "quant":
            return dict(op=op, rows=rows, k=k, type=rng.choice(["f32", "f16", "bf16"]))
        return dict(op=op, rows=rows, k=k, residual=rng.randint(0, 1))
    if op == "gemm":
        m, k = _log_int(rng, 16, 16384), 32 * _log_int(rng, 1, 512)
        most = max(1, min(4096, 14336 * 4096 * 2048 // (m * k), 14336 * 2048 // m))
        return dict(op=op, m=m, k=k, n=_log_int(rng, 1, most), scaled=rng.randint(0, 1))
    if op == "append":
        n_kv, head_dim = rng.choice([1, 2, 3, 4, 8, 16]), 32 * rng.randint(1, 8)
        most = max(1, 8192 * 8 * 128 // (n_kv * head_dim))
        return dict(op=op, tokens=_log_int(rng, 1, min(8192, most)), run=_log_int(rng, 1, 1024), n_kv=n_kv,
                    group=rng.randint(1, 8), head_dim=head_dim, page=rng.choice([1, 8, 16, 32, 64, 128]),
                    layout=rng.choice(["hnd", "nhd"]), pad=rng.randint(0, 9))
    n_kv, head_dim, batch = rng.choice([1, 2, 3, 4, 8, 16]), 32 * rng.randint(1, 8), _log_int(rng, 1, 64)
    most = max(1, 48 * 8192 * 8 * 128 // (n_kv * head_dim * batch))
    return dict(op=op, batch=batch, max_len=_log_int(rng, 1, min(65536, most)), n_kv=n_kv,
                group=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 20]), head_dim=head_dim,
                page=rng.choice([1, 8, 16, 32, 64, 128]), layout=rng.choice(["hnd", "nhd"]), even=rng.randint(0, 1),
                pad=rng.randint(0, 3))


def _lens(case):
    n, most = case["batch"], case["max_len"]
    full = [most] * n if case["even"] else [max(1, int(round(most * ((i + 1) / n) ** 2))) for i in range(n)]
    return full + [0] * case["pad"]


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["k"]
        return {"bytes": n * (4.0 + 2 * MX_BYTES + (4 if case["type"] == "f32" else 2)), "flops": 3.0 * n}
    if op == "norm":  # the codes are read back: the values are the case's output
        n = case["rows"] * case["k"]
        return {"bytes": n * (8.0 + 2 * MX_BYTES + (8 if case["residual"] else 0)) + 4.0 * (case["k"] + case["rows"]),
                "flops": 8.0 * n}
    if op == "gemm":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": (m + n) * k * MX_BYTES + 4.0 * m * n + 4.0 * n * case["scaled"], "flops": 2.0 * m * n * k}
    if op == "append":  # the whole cache is read back: its values are the case's output
        n, row = case["tokens"], case["n_kv"] * case["head_dim"]
        run_ = min(case["run"], n)
        places = (-(-n // run_) * -(-run_ // case["page"]) + 4) * case["page"]
        return {"bytes": 2.0 * row * (n * (4 + MX_BYTES) + places * (4 + MX_BYTES)) + 4.0 * (n + case["pad"]),
                "flops": 6.0 * n * row}
    lens, hq, d = _lens(case), case["n_kv"] * case["group"], case["head_dim"]
    kv = sum(lens) * case["n_kv"] * d
    pages = sum(-(-n // case["page"]) for n in lens)
    return {"bytes": 2 * kv * MX_BYTES + len(lens) * (8.0 * hq * d + 4 * hq + 4) + 4.0 * pages,
            "flops": 4.0 * kv * case["group"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _activations(g, rows, k):
    """Normal values with a few channels some times larger than the rest, as activations have them."""
    channel = torch.where(torch.rand(k, generator=g, device="cuda") < 0.02, 8.0, 1.0)
    return _randn(g, rows, k) * channel


def _random_mx(g, *shape):
    """Random codes and scales of values of size about one, without their float form (large)."""
    k = shape[-1]
    codes = torch.randint(0, 256, shape[:-1] + (k // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(124, 128, shape[:-1] + (k // 32,), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def _pages(g, case, n_pages, filled):
    """An empty (or filled) cache: codes and scales of keys and values in the order of `layout`."""
    hnd = case["layout"] == "hnd"
    shape = (n_pages, case["n_kv"], case["page"]) if hnd else (n_pages, case["page"], case["n_kv"])
    d, out = case["head_dim"], {}
    for name in ("k", "v"):
        if filled:
            out[name], out[name + "s"] = _random_mx(g, *shape, d)
        else:
            out[name] = torch.zeros(shape + (d // 2,), dtype=torch.uint8, device="cuda")
            out[name + "s"] = torch.zeros(shape + (d // 32,), dtype=torch.uint8, device="cuda")
    return out


def _views(case, cache):
    """[n_pages, n_kv, page, ..] views of the cache's tensors."""
    return {n: t if case["layout"] == "hnd" else t.transpose(1, 2) for n, t in cache.items()}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    state = {"case": case, "seed": seed}
    if op == "quant":
        x = _activations(g, case["rows"], case["k"]).to(DTYPES[case["type"]])
        state |= {"x": x, "q": torch.empty(case["rows"], case["k"] // 2, dtype=torch.uint8, device="cuda"),
                  "e": torch.empty(case["rows"], case["k"] // 32, dtype=torch.uint8, device="cuda"),
                  "out": torch.empty(case["rows"], case["k"], device="cuda")}
    elif op == "norm":
        n, k = case["rows"], case["k"]
        state |= {"x": _randn(g, n, k), "r": 3 * _randn(g, n, k) if case["residual"] else None,
                  "w": 1 + 0.2 * _randn(g, k), "h": torch.empty(n, k, device="cuda") if case["residual"] else None,
                  "q": torch.empty(n, k // 2, dtype=torch.uint8, device="cuda"),
                  "e": torch.empty(n, k // 32, dtype=torch.uint8, device="cuda"),
                  "s": torch.empty(n, device="cuda"), "out": torch.empty(n, k, device="cuda")}
    elif op == "gemm":
        m, k, n = case["m"], case["k"], case["n"]
        wq, we = _pack(_plain_codes(_randn(g, m, k) * k ** -0.5))
        xq, xe = _pack(_plain_codes(_activations(g, n, k)))
        s = torch.rand(n, generator=g, device="cuda") + 0.5 if case["scaled"] else None
        state |= {"wq": wq, "we": we, "xq": xq, "xe": xe, "s": s, "out": torch.empty(n, m, device="cuda")}
    elif op == "append":
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
                  "slots": torch.cat([slots, slots.new_full((case["pad"],), -1)]).int(),
                  "out": {n_: torch.empty(cache[n_].shape[:-1] + (d,), device="cuda") for n_ in ("k", "v")}}
    else:
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
    if own and op in ("append", "attend"):
        import gemv_prefill_decode_amd as qmm

        c = _views(case, state["cache"])
        state["handle"] = qmm.KVCache(c["k"], c["v"], c["ks"], c["vs"])
    return state


# ------------------------------------------------------------------ plain forms
def _pow2(n):
    """2^n as float32 for whole n in [-126, 127], from its bits."""
    return ((n + 127) << 23).view(torch.float32)


def _plain_codes(z):
    """(codes, scale bytes), int32, of float32 rows in runs of 32."""
    z = z.float().unflatten(-1, (-1, 32))
    top = z.abs().amax(-1, keepdim=True)
    bad = ~(top < math.inf)
    exponent = torch.frexp(torch.where(bad, torch.zeros_like(top), top)).exponent  # top in [2^(exponent-1), 2^exponent)
    e = torch.where(top == 0, -127, exponent - 3).clamp(min=-127)
    a = z.abs() * _pow2((-e).int())
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = torch.where(bad, 0, code + 8 * torch.signbit(z))
    return code.flatten(-2).int(), torch.where(bad, 255, e + 127).squeeze(-1).int()


def _pack(coded):
    codes, scales = coded
    return (codes[..., ::2] + 16 * codes[..., 1::2]).to(torch.uint8), scales.to(torch.uint8)


def _plain_values(q, e):
    """float32 values of packed codes and their scale bytes."""
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    pairs = torch.stack([t.repeat(16), t.repeat_interleave(16)], dim=1)      # a byte's low, then its high nibble
    x = pairs.index_select(0, q.reshape(-1).int()).reshape(e.shape + (32,))
    e = e.int().unsqueeze(-1)
    x = x * _pow2((e - 127).clamp(-126, 127)) * torch.where(e == 0, 0.5, 1.0)
    return torch.where(e == 255, math.nan, x).flatten(-2)


def _plain_quant(s):
    return _plain_values(*_pack(_plain_codes(s["x"])))


def _plain_norm(s):
    h = s["x"] if s["r"] is None else s["x"] + s["r"]
    inv = torch.rsqrt((h * h).mean(-1) + EPS)
    more = {} if s["r"] is None else {"h": h}
    # 1/rms is one factor of a whole row, kept apart: the codes are those of h*w
    return {"y": _plain_values(*_pack(_plain_codes(h * s["w"]))), "s": inv, **more}


def _plain_gemm(s):
    out = _plain_values(s["xq"], s["xe"]) @ _plain_values(s["wq"], s["we"]).T
    return out if s["s"] is None else out * s["s"][:, None]


def _cache_values(c):
    return {"k": _plain_values(c["k"], c["ks"]), "v": _plain_values(c["v"], c["vs"])}


def _plain_append(s):
    case, c = s["case"], _views(s["case"], s["cache"])
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    page, at = slots // case["page"], slots % case["page"]
    for new, n in ((s["knew"], "k"), (s["vnew"], "v")):
        c[n][page, :, at], c[n + "s"][page, :, at] = _pack(_plain_codes(new[live]))
    return _cache_values(s["cache"])


def _plain_gather(codes, scales, table):
    """The cache's rows of every sequence in order: float32 [batch, n_kv, width * page, head_dim]."""
    return _plain_values(codes[table].transpose(1, 2).flatten(2, 3), scales[table].transpose(1, 2).flatten(2, 3))


def _plain_attend(s):
    case, c = s["case"], _views(s["case"], s["cache"])
    b, hq, d = s["q"].shape
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    table = s["table"].long().clamp(min=0)
    tokens = table.shape[1] * case["page"]
    step = max(1, (1 << 31) // (tokens * case["n_kv"] * d * 4))      # sequences at a time: some GB of float rows
    for i in range(0, b, step):
        rows = slice(i, i + step)
        q = s["q"][rows].reshape(-1, case["n_kv"], case["group"], d)
        dead = torch.arange(tokens, device="cuda") >= s["lens"][rows, None]
        score = (q @ _plain_gather(c["k"], c["ks"], table[rows]).transpose(-1, -2)) * d ** -0.5
        score = score.masked_fill(dead[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        v = _plain_gather(c["v"], c["vs"], table[rows]).masked_fill(dead[:, None, :, None], 0.0)
        out[rows] = ((p @ v) / torch.where(total == 0, torch.ones_like(total), total)).reshape(-1, hq, d)
        lse[rows] = (top + torch.log(total)).reshape(-1, hq)
    return {"out": out, "lse": lse}


PLAIN = {"quant": _plain_quant, "norm": _plain_norm, "gemm": _plain_gemm, "append": _plain_append, "attend": _plain_attend}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import gemv_prefill_decode_amd as qmm

    op = s["case"]["op"]
    if op == "quant":
        qmm.quantize_mxfp4(s["x"], q=s["q"], e=s["e"])
        return qmm.dequantize_mxfp4(s["q"], s["e"], out=s["out"])
    if op == "norm":
        qmm.add_rmsnorm_mxfp4(s["x"], s["w"], s["r"], eps=EPS, q=s["q"], e=s["e"], s=s["s"], h=s["h"])
        more = {} if s["r"] is None else {"h": s["h"]}
        return {"y": qmm.dequantize_mxfp4(s["q"], s["e"], out=s["out"]), "s": s["s"], **more}
    if op == "gemm":
        return qmm.gemm_mxfp4(s["wq"], s["we"], s["xq"], s["xe"], x_scale=s["s"], out=s["out"])
    if op == "append":
        qmm.kv_append(s["handle"], s["knew"], s["vnew"], s["slots"])
        c = s["cache"]
        return {n: qmm.dequantize_mxfp4(c[n], c[n + "s"], out=s["out"][n]) for n in ("k", "v")}
    qmm.paged_attention(s["q"], s["handle"], s["table"], s["lens"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_round(x):
    """The values that x's codes and scales stand for, float64: the nearest of the grid in runs of
    32, ties to the even code. Which code is nearest is decided without rounding."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2
    # log2 of a value just below a power of two may round up to it
    e = torch.where(top < torch.pow(2.0, e + 2), e - 1, e).clamp(min=-127)
    unit = torch.pow(2.0, e)
    a, best = x.abs() / unit, torch.zeros_like(x)
    for i in range(1, 8):
        up = 2 * a - (GRID[i - 1] + GRID[i])
        best = torch.where((up > 0) | ((up == 0) & (i % 2 == 0)), GRID[i], best)
    return (torch.sign(x) * best * unit).flatten(-2)


def _exact_decode(q, e):
    """float64 values, from the bits of each code."""
    c = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)
    mantissa, exponent = (c & 1).double(), ((c >> 1) & 3).double()
    a = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.pow(2.0, exponent - 1))
    a = torch.where(c >= 8, -a, a)
    return a * torch.pow(2.0, e.double() - 127).repeat_interleave(32, dim=-1)


def _exact_norm(s):
    h32 = s["x"] if s["r"] is None else s["x"] + s["r"]
    h = h32.double()
    more = {} if s["r"] is None else {"h": s["x"].double() + s["r"].double()}
    # codes follow the float32 products: their rounding decides a tie
    return {"y": _exact_round(h32 * s["w"]), "s": 1 / torch.sqrt(h.pow(2).sum(-1) / h.shape[1] + EPS), **more}


def _exact_gemm(s):
    out = torch.mm(_exact_decode(s["xq"], s["xe"]), _exact_decode(s["wq"], s["we"]).T.contiguous())
    return out if s["s"] is None else out * s["s"].double()[:, None]


def _exact_append(s):
    case, at, out = s["case"], s["slots"].tolist(), {}
    live = [i for i, slot in enumerate(at) if slot >= 0]
    page, place = (torch.tensor([f(at[i], case["page"]) for i in live], device="cuda") for f in (lambda a, b: a // b, lambda a, b: a % b))
    for n, new in (("k", s["knew"]), ("v", s["vnew"])):
        c = s["cache"][n]
        whole = torch.zeros(c.shape[:-1] + (case["head_dim"],), dtype=torch.float64, device="cuda")
        rows = _exact_round(new.contiguous())[live]
        if case["layout"] == "hnd":
            whole[page, :, place] = rows
        else:
            whole[page, place] = rows
        out[n] = whole
    return out


def _exact_attend(s):
    case, ps = s["case"], s["case"]["page"]
    b, hq, d = s["q"].shape
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        page, at = s["table"][i].long()[t // ps], t % ps
        for h in range(case["n_kv"]):
            place = (page, h, at) if case["layout"] == "hnd" else (page, at, h)
            k, v = (_exact_decode(s["cache"][x][place], s["cache"][x + "s"][place]) for x in ("k", "v"))
            mine = slice(h * case["group"], (h + 1) * case["group"])
            score = torch.mm(s["q"][i, mine].double(), k.T.contiguous()) / math.sqrt(d)
            lse[i, mine] = torch.logsumexp(score, -1)
            out[i, mine] = torch.mm(torch.exp(score - lse[i, mine][:, None]), v)
    return {"out": out, "lse": lse}


EXACT = {"quant": lambda s: _exact_round(s["x"]), "norm": _exact_norm, "gemm": _exact_gemm, "append": _exact_append,
         "attend": _exact_attend}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
