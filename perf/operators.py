"""What is measured of the decoder-step operators: the cases, their inputs, their plain forms.

The operators are those that run between the quantized linear layers of a speculative
decoder's step: the residual + RMS norm (bfloat16, 8-bit or 4-bit output), the paged
key/value cache (written quantized, read back), attention of a chunk of new tokens over that
cache, and sampling.  With `own` false, run() computes them with elementary torch operations
in 32 bits (64 for the norm's sum and the sampling weights); with `own` true it calls the
framework.  exact() evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

# head layouts: the Qwen2.5-1.5B, Qwen2.5-7B and Llama-2-7B shapes, and generic ones
_HEADS = [(12, 2), (28, 4), (32, 32), (32, 8), (16, 16), (8, 1)]


# ------------------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one token of a Qwen2.5-1.5B-shaped draft: the call is all latency
        dict(name="norm-draft-m1", op="norm", m=1, h=1536, x="bf16", res="bf16", bits=16),
        # the norm ahead of a 4-bit-activation product: Llama-2-7B draft at batch 32
        dict(name="norm-a4-m32", op="norm", m=32, h=4096, x="f32", res="bf16", bits=4),
        # a long prompt's rows straight from the float32 product, 8-bit output
        dict(name="norm-prompt-m8192", op="norm", m=8192, h=3584, x="f32", res="bf16", bits=8),
        # five verified tokens enter an 8-bit cache from a fused float32 qkv product
        dict(name="kv-verify-t5", op="kv_write", t=5, hkv=4, d=128, page=64, cache=8, src="f32"),
        # a prompt enters the cache of a 32-head model
        dict(name="kv-prompt-t8191", op="kv_write", t=8191, hkv=32, d=128, page=64, cache=8, src="bf16"),
        # a cached prefix is read back as bfloat16
        dict(name="kv-readback-t30000", op="kv_read", t=30000, hkv=4, d=128, page=16, cache=8, out="bf16"),
        # one draft token over a short context, 16-bit cache
        dict(name="attn-draft-b1", op="attn", b=1, n=1, ctx=777, hq=12, hkv=2, d=128, page=16, cache=16),
        # gamma + 1 = 5 tokens verified over a long context, 8-bit cache
        dict(name="attn-verify-b1", op="attn", b=1, n=5, ctx=16387, hq=28, hkv=4, d=128, page=64, cache=8),
        # batched verify: 32 sequences of different lengths, 5 tokens each, 32 key/value heads
        dict(name="attn-verify-b32", op="attn", b=32, n=5, ctx=4096, hq=32, hkv=32, d=128, page=64, cache=16),
        # a 2048-token piece of a prompt over what is cached of it
        dict(name="attn-prompt-n2048", op="attn", b=1, n=2048, ctx=8000, hq=28, hkv=4, d=128, page=64, cache=16),
        # one draft token drawn from a large vocabulary
        dict(name="sample-draft-b1", op="sample", b=1, v=152064, kind="f32", k=1, p=1, mp=0),
        # every verified position of a batch of 32 drawn, the rows' settings mixed
        dict(name="sample-verify-b160", op="sample", b=160, v=152064, kind="f32", k=1, p=1, mp=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "kv_write", "kv_read", "attn", "attn", "sample"])
    if op == "norm":
        bits = rng.choice([16, 16, 8, 4])
        h = 128 * _log_int(rng, 6, 64)
        if h == 3072:
            h += 128
        if bits == 16 and rng.random() < 0.4:
            h -= rng.randrange(1, 100)
        m = min(_log_int(rng, 1, 8192), 8192 * 3584 // h)
        return dict(op=op, m=m, h=h, x=rng.choice(["f32", "bf16"]), res=rng.choice(["f32", "bf16", "none"]), bits=bits)
    if op in ("kv_write", "kv_read"):
        hkv, d = rng.choice([1, 2, 4, 8, 32]), rng.choice([64, 128])
        t = min(_log_int(rng, 1, 32768), 8191 * 32 * 128 // (hkv * d))
        c = dict(op=op, t=t, hkv=hkv, d=d, page=rng.choice([16, 32, 48, 64, 128]), cache=rng.choice([8, 8, 16]))
        if op == "kv_write":
            c["src"] = rng.choice(["f32", "bf16"])
        else:
            c["out"] = rng.choice(["f32", "bf16"])
        return c
    if op == "attn":
        hq, hkv = rng.choice(_HEADS)
        d = rng.choice([64, 128, 128])
        n = rng.choice([1, rng.randrange(2, 9), _log_int(rng, 1, 2048)])
        b, ctx = _log_int(rng, 1, 48), _log_int(rng, 1, 32768)
        # no more bytes of cache, scores or products than the listed cases
        b = max(1, min(b, 32 * 4096 * 32 * 128 // (ctx * hkv * d), 2048 * 8000 * 28 // (n * ctx * hq)))
        n = max(1, min(n, 2048 * 8000 * 28 // (b * ctx * hq)))
        return dict(op=op, b=b, n=n, ctx=ctx, hq=hq, hkv=hkv, d=d, page=rng.choice([16, 32, 48, 64, 128]), cache=rng.choice([8, 16]))
    v = _log_int(rng, 500, 160000)
    if v == 3072:
        v += 1
    return dict(op=op, b=min(_log_int(rng, 1, 192), 160 * 152064 // v), v=v, kind=rng.choice(["f32", "f32", "bf16"]),
                k=rng.choice([0, 1]), p=rng.choice([0, 1]), mp=rng.choice([0, 1]))


# ------------------------------------------------------------------------------------
# Inputs

def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _lengths(c):
    """The sequences' total lengths and chunk lengths: ragged over a batch, the first the longest."""
    kv = [max(1, c["ctx"] - (i * c["ctx"] * 5 // (c["b"] * 8))) if i else c["ctx"] for i in range(c["b"])]
    n = [min(c["n"] if i % 4 != 3 else max(1, c["n"] - i % 3), kv[i]) for i in range(c["b"])]
    return kv, n


def _quantized(shape, gen):
    """8-bit codes and scales as the write leaves them: the largest code of each row near 127."""
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = codes.view(shape[0], -1)
    step = max(1, (1 << 26) // flat.shape[1])
    for i in range(0, shape[0], step):
        part = torch.randn(flat[i:i + step].shape, generator=gen, device="cuda")
        flat[i:i + step] = part.mul_(46.0).round_().clamp_(-127, 127).to(torch.int8)
    scales = torch.rand(shape[:-1], generator=gen, device="cuda").mul_(0.012).add_(0.016)
    return codes, scales


def _half(shape, gen):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 26) // flat.shape[1])
    for i in range(0, shape[0], step):
        flat[i:i + step] = torch.randn(flat[i:i + step].shape, generator=gen, device="cuda").to(torch.bfloat16)
    return out


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "norm":
        # a residual stream with a few large channels, the product's rows added to it
        big = 1 + 20 * (torch.rand(c["h"], generator=gen, device="cuda") < 0.01).float()
        s["x"] = torch.randn(c["m"], c["h"], generator=gen, device="cuda").to(_dtype(c["x"]))
        s["res"] = None
        if c["res"] != "none":
            s["res"] = (2 * big * torch.randn(c["m"], c["h"], generator=gen, device="cuda")).to(_dtype(c["res"]))
        s["w"] = (1 + 0.2 * torch.randn(c["h"], generator=gen, device="cuda")).to(torch.bfloat16)
    elif c["op"] == "kv_write":
        pages = c["t"] // c["page"] + 2
        # keys and values are slices of one fused qkv row, as a product leaves them
        qkv = torch.randn(c["t"], 3 * c["hkv"], c["d"], generator=gen, device="cuda").to(_dtype(c["src"]))
        s["k"], s["v"] = qkv[:, c["hkv"]:2 * c["hkv"]], qkv[:, 2 * c["hkv"]:]
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(c["t"], device="cuda") + c["page"] // 3  # the chunk begins inside a page
        s["slots"] = order[at // c["page"]] * c["page"] + at % c["page"]
        _caches(s, pages, gen)
    elif c["op"] == "kv_read":
        pages = -(-c["t"] // c["page"]) + 1
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(c["t"], device="cuda")
        s["slots"] = order[at // c["page"]] * c["page"] + at % c["page"]
        _caches(s, pages, gen)
    elif c["op"] == "attn":
        kv, n = _lengths(c)
        width = -(-max(kv) // c["page"])
        used = [-(-length // c["page"]) for length in kv]
        pages = sum(used) + 1
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros(c["b"], width, dtype=torch.int32, device="cuda")
        at = 0
        for i, u in enumerate(used):
            table[i, :u] = order[at:at + u]
            at += u
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        # the queries are a slice of the fused qkv rows
        qkv = torch.randn(starts[-1], c["hq"] + 2 * c["hkv"], c["d"], generator=gen, device="cuda").mul_(1.5)
        s["q"] = qkv.to(torch.bfloat16)[:, :c["hq"]]
        s["table"] = table
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["max_q"], s["max_kv"] = max(n), max(kv)
        _caches(s, pages, gen)
    else:
        # most of a vocabulary is noise; a few dozen tokens stand out
        z = 2.0 * torch.randn(c["b"], c["v"], generator=gen, device="cuda")
        some = torch.randint(0, c["v"], (c["b"], 48), generator=gen, device="cuda")
        lift = torch.rand(c["b"], 48, generator=gen, device="cuda").log_().mul_(-3.0).add_(7.0)
        s["logits"] = z.scatter_(1, some, lift).to(_dtype(c["kind"]))
        rows = lambda: torch.rand(c["b"], generator=gen, device="cuda")  # noqa: E731
        t = 0.6 + 0.6 * rows()
        s["t"] = torch.where(rows() < 0.06 * (c["b"] > 1), torch.zeros_like(t), t)  # some rows are greedy
        s["k"] = s["p"] = s["mp"] = None
        if c["k"]:
            s["k"] = torch.where(rows() < 0.2 * (c["b"] > 1), torch.zeros_like(t), 10 + 90 * rows()).to(torch.int32)
        if c["p"]:
            s["p"] = torch.where(rows() < 0.1 * (c["b"] > 1), torch.ones_like(t), 0.7 + 0.28 * rows())
        if c["mp"]:
            s["mp"] = torch.where(rows() < 0.5, torch.zeros_like(t), 0.1 * rows())
        s["u"] = rows()
    return s


def _caches(s, pages, gen):
    c = s["c"]
    shape = (pages, c["hkv"], c["page"], c["d"])
    if c["cache"] == 8:
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _quantized(shape, gen), _quantized(shape, gen)
    else:
        s["kc"], s["vc"], s["ks"], s["vs"] = _half(shape, gen), _half(shape, gen), None, None


# ------------------------------------------------------------------------------------
# One pass

_EPS = 1e-6


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import int4_weight_only_gemm_amd as w4
    c = s["c"]
    if c["op"] == "norm":
        r = w4.rms_norm(s["x"], s["w"], residual=s["res"], eps=_EPS, bits=c["bits"])
        if c["bits"] != 16:  # the values that codes and scales stand for
            y = w4.dequantize_activations(r[0], r[1], bits=c["bits"])
            return (y,) + tuple(r[2:])
        return r
    if c["op"] == "kv_write":
        w4.kv_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        return w4.kv_read(s["slots"], s["kc"], s["vc"], s["ks"], s["vs"], dtype=torch.float32)
    if c["op"] == "kv_read":
        return w4.kv_read(s["slots"], s["kc"], s["vc"], s["ks"], s["vs"], dtype=_dtype(c["out"]))
    if c["op"] == "attn":
        return w4.paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["q_start"], s["kv_len"],
                                  s["max_q"], s["max_kv"], s["ks"], s["vs"])
    return w4.sample(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["mp"])


def _run_plain(s):
    return {"norm": _plain_norm, "kv_write": _plain_write, "kv_read": _plain_read, "attn": _plain_attn,
            "sample": _plain_sample}[s["c"]["op"]](s)


def _codes(x, most, least):
    """Symmetric codes of the last axis and their scale, in 32 bits."""
    top = x.abs().amax(-1, keepdim=True)
    scale = top / torch.full_like(top, most)  # a division by a number would be a product with its reciprocal
    return torch.where(scale > 0, (x / scale).round().clamp(least, most), torch.zeros_like(x)), scale


def _plain_norm(s):
    c = s["c"]
    r = s["x"]
    if s["res"] is not None:
        r = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    f = r.float()
    inv = (1 / (f.double().square().mean(-1, keepdim=True) + _EPS).sqrt()).float()
    y = f * inv * s["w"].float()
    if c["bits"] == 16:
        y = y.to(torch.bfloat16)
        return y if s["res"] is None else (y, r)
    groups = y.view(c["m"], -1, 128)
    if c["bits"] == 8:
        q, scale = _codes(groups, 127, -127)
    else:
        q, scale = _codes(groups.to(torch.bfloat16).float(), 7, -8)
    y = (q * scale).view(c["m"], c["h"])
    return (y,) if s["res"] is None else (y, r)


def _take(cache, scale, slots, page):
    v = cache[slots // page, :, slots % page].float()
    return v if scale is None else v * scale[slots // page, :, slots % page].unsqueeze(-1)


def _plain_write(s):
    at, off = s["slots"] // s["c"]["page"], s["slots"] % s["c"]["page"]
    for x, cache, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        if scales is None:
            cache[at, :, off] = x.to(cache.dtype)
        else:
            q, scale = _codes(x.float(), 127, -127)
            cache[at, :, off] = q.to(torch.int8)
            scales[at, :, off] = scale.squeeze(-1)
    return (_take(s["kc"], s["ks"], s["slots"], s["c"]["page"]), _take(s["vc"], s["vs"], s["slots"], s["c"]["page"]))


def _plain_read(s):
    kind = _dtype(s["c"]["out"])
    return (_take(s["kc"], s["ks"], s["slots"], s["c"]["page"]).to(kind),
            _take(s["vc"], s["vs"], s["slots"], s["c"]["page"]).to(kind))


def _dense(cache, scale, table):
    """[B, Hkv, width * page, D] in 32 bits."""
    at = table.long()
    x = cache[at].float()
    if scale is not None:
        x = x * scale[at].unsqueeze(-1)
    b, w, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, w * p, d)


def _plain_attn(s):
    c = s["c"]
    b, hq, hkv, d, n = c["b"], c["hq"], c["hkv"], c["d"], s["max_q"]
    k, v = _dense(s["kc"], s["ks"], s["table"]), _dense(s["vc"], s["vs"], s["table"])
    start, kv = s["q_start"][:-1].long(), s["kv_len"].long()
    count = s["q_start"][1:].long() - start
    i = torch.arange(n, device="cuda")
    rows = (start[:, None] + i).clamp_(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(b, hkv, hq // hkv, n, -1) * (1 / math.sqrt(d))
    at = (kv - count)[:, None] + i
    j = torch.arange(k.shape[2], device="cuda")
    sees = (j <= at[..., None]) & (j < kv[:, None, None])
    score = score.masked_fill(~sees[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = (score - torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp()
    total = e.sum(-1, keepdim=True)
    v = v.masked_fill((j >= kv[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(e.view(b, hkv, -1, k.shape[2]), v).view(b, hkv, hq // hkv, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d).to(torch.bfloat16)
    return o[i < count[:, None]]


def _plain_sample(s):
    c = s["c"]
    z = s["logits"].float()
    order = z.sort(dim=-1, descending=True, stable=True)
    greedy = (s["t"] <= 0)[:, None]
    t = torch.where(greedy, torch.ones_like(s["t"])[:, None], s["t"][:, None]).double()
    w = ((order.values.double() - order.values[:, :1].double()) / t).exp()
    rank = torch.arange(c["v"], device="cuda")
    keep = ~greedy | (rank < 1)
    if s["k"] is not None:
        keep = keep & ((s["k"] <= 0)[:, None] | (rank < s["k"][:, None]))
    w = w * keep
    if s["p"] is not None:
        before = w.cumsum(-1) - w
        keep = keep & ((s["p"] >= 1)[:, None] | (rank < 1) | (before < s["p"][:, None].double() * w.sum(-1, keepdim=True)))
    if s["mp"] is not None:
        keep = keep & (w >= s["mp"][:, None].double())
    w = torch.zeros_like(w).scatter_(1, order.indices, w * keep)  # back in the order of the vocabulary
    total = w.sum(-1, keepdim=True)
    token = ((w.cumsum(-1) > s["u"][:, None].double() * total) & (w > 0)).to(torch.int8).argmax(-1, keepdim=True)
    return token.squeeze(-1).to(torch.int32), (w.gather(1, token) / total).squeeze(-1).float()


# ------------------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    c = case
    if c["op"] == "norm":
        size = {"f32": 4, "bf16": 2, "none": 0}
        out = {16: 2.0, 8: 4.0, 4: 4.0}[c["bits"]]  # 8 and 4 bits: as the values that are returned
        return {"bytes": c["m"] * c["h"] * (size[c["x"]] + 2 * size[c["res"]] + out) + 2 * c["h"], "flops": 6 * c["m"] * c["h"]}
    if c["op"] in ("kv_write", "kv_read"):
        rows = 2 * c["t"] * c["hkv"]
        held = c["d"] + 4 if c["cache"] == 8 else 2 * c["d"]
        if c["op"] == "kv_write":
            return {"bytes": rows * (c["d"] * {"f32": 4, "bf16": 2}[c["src"]] + held + 4 * c["d"]) + 8 * c["t"], "flops": 4 * rows * c["d"]}
        return {"bytes": rows * (held + c["d"] * {"f32": 4, "bf16": 2}[c["out"]]) + 8 * c["t"], "flops": rows * c["d"]}
    if c["op"] == "attn":
        kv, n = _lengths(c)
        held = c["d"] + 4 if c["cache"] == 8 else 2 * c["d"]
        pairs = sum(x * length - x * (x - 1) // 2 for length, x in zip(kv, n))
        return {"bytes": 2 * sum(kv) * c["hkv"] * held + 4 * sum(n) * c["hq"] * c["d"], "flops": 4 * c["d"] * c["hq"] * pairs}
    return {"bytes": c["b"] * c["v"] * {"f32": 4, "bf16": 2}[c["kind"]], "flops": 4 * c["b"] * c["v"]}


# ------------------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence and row by row

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        r = s["x"].double()
        if s["res"] is not None:
            r = r + s["res"].double()
            stored = r.to(s["res"].dtype).double()  # the norm is of the residual as it is kept
        else:
            stored = r
        root = (torch.linalg.vector_norm(stored, dim=1) ** 2 / c["h"] + _EPS).sqrt()[:, None]
        if c["bits"] == 16:
            y = stored / root * s["w"].double()
        else:
            # which code a value takes is defined by binary32 steps: each is the 64-bit result, rounded
            y = _step(_step(stored * _step(1 / root)) * s["w"].double())
            y = y.to(torch.bfloat16).double() if c["bits"] == 4 else y
            y = torch.cat([_grid(g, 7 if c["bits"] == 4 else 127) for g in y.split(128, 1)], 1)
        if s["res"] is None:
            return y if c["bits"] == 16 else (y,)
        return y, r
    if c["op"] == "kv_write":
        if c["cache"] == 8:
            return tuple(_grid(x.double(), 127) for x in (s["k"], s["v"]))
        return tuple(x.to(torch.bfloat16).double() for x in (s["k"], s["v"]))  # as they are kept
    if c["op"] == "kv_read":
        out = []
        for cache, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            x = cache.transpose(1, 2).reshape(-1, c["hkv"], c["d"]).index_select(0, s["slots"]).double()
            if scale is not None:
                x = x * scale.transpose(1, 2).reshape(-1, c["hkv"]).index_select(0, s["slots"]).double()[..., None]
            out.append(x)
        return tuple(out)
    if c["op"] == "attn":
        return _exact_attn(c, s)
    return _exact_sample(c, s)


def _step(x):
    return x.float().double()


def _grid(x, most):
    unit = _step(x.abs().max(-1, keepdim=True).values / most)
    return torch.nan_to_num(_step(x / unit)).round() * unit


def _exact_attn(c, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    kv, n = _lengths(c)
    per, at = c["hq"] // c["hkv"], 0
    for i in range(c["b"]):
        pages = s["table"][i, :-(-kv[i] // c["page"])].long()
        for h in range(c["hkv"]):
            k, v = (x[pages, h].reshape(-1, c["d"])[:kv[i]].double() for x in (s["kc"], s["vc"]))
            if s["ks"] is not None:
                k, v = (x * y[pages, h].reshape(-1, 1)[:kv[i]].double() for x, y in ((k, s["ks"]), (v, s["vs"])))
            hidden = torch.ones(n[i], kv[i], dtype=torch.bool, device="cuda").triu_(kv[i] - n[i] + 1)
            for g in range(h * per, (h + 1) * per):
                score = (s["q"][at:at + n[i], g].double() @ k.t()) / math.sqrt(c["d"])
                out[at:at + n[i], g] = torch.softmax(score.masked_fill_(hidden, -math.inf), -1) @ v
        at += n[i]
    return out


def _exact_sample(c, s):
    tokens, probs = [], []
    for i in range(c["b"]):
        z = s["logits"][i].double()
        t = float(s["t"][i])
        if t <= 0:
            tokens.append(int((z == z.max()).nonzero()[0]))
            probs.append(1.0)
            continue
        by = torch.argsort(z, descending=True, stable=True)
        if s["k"] is not None and int(s["k"][i]) > 0:
            by = by[:int(s["k"][i])]
        w = torch.softmax(z[by] / t, 0)
        if s["p"] is not None and float(s["p"][i]) < 1:
            first = int((w.cumsum(0) >= float(s["p"][i])).to(torch.int8).argmax())
            by, w = by[:first + 1], w[:first + 1]
        if s["mp"] is not None:
            kept = w >= float(s["mp"][i]) * w[0]
            by, w = by[kept], w[kept]
        by, back = by.sort()
        w = w[back] / w.sum()
        at = min(int((w.cumsum(0) <= float(s["u"][i])).sum()), len(w) - 1)
        tokens.append(int(by[at]))
        probs.append(float(w[at]))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)
