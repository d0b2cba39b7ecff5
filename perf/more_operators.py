"""Cases of the serving step around a paged cache of latent vectors.

Latent attention caches one vector of 512 latent and 64 rotary elements a token,
shared by all heads.  Five operators, each in its plain form (elementary torch
operations in fp32) and, where `own` is set, as the calls a user makes of the
library:

  query    a head's 128 query elements into the latent space (the head's key
           up-projection absorbed into the query), the 64 rotary ones turned
  append   RMS norm of new tokens' latent part, rotation of the rotary part,
           both into their pages
  decode   attention of one or a few new tokens a sequence over the pages
  output   the attended latent vectors back to 128 value elements a head
  gather   rows of the cache back as the ragged tensors that a prefill over
           expanded keys and values starts from

Pages are [num_pages, 64, 576], 512 latent elements first.
"""
import math
import random

import torch

own = False

PAGE = 64
LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
ROW = LATENT + ROPE
DEV = "cuda"
MAX_POS = 32768
SCALE = (NOPE + ROPE) ** -0.5
T16 = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence, all heads: the latency of a step's first product
        {"name": "query token", "op": "query", "tokens": 1, "heads": 128, "interleaved": False, "dtype": "bf16"},
        # one decode step of a batch of 64
        {"name": "query step", "op": "query", "tokens": 64, "heads": 128, "interleaved": False, "dtype": "bf16"},
        # a chunk of prompts with half of the heads, an odd number of tokens, the other pairing
        {"name": "query chunk", "op": "query", "tokens": 1999, "heads": 64, "interleaved": True, "dtype": "f16"},
        # one decode step of a batch of 64
        {"name": "append step", "op": "append", "batch": 64, "new": 1, "prefix": 4096, "interleaved": False, "dtype": "bf16"},
        # chunks of sixteen prompts
        {"name": "append chunk", "op": "append", "batch": 16, "new": 1024, "prefix": 8192, "interleaved": True, "dtype": "bf16"},
        # one short sequence: the latency of an attention call
        {"name": "decode one", "op": "decode", "batch": 1, "shortest": 777, "longest": 777, "heads": 128, "new": 1, "dtype": "bf16"},
        # the decode batch: 64 sequences of 1 to 4096 keys, all heads
        {"name": "decode batch", "op": "decode", "batch": 64, "shortest": 1, "longest": 4096, "heads": 128, "new": 1, "dtype": "bf16"},
        # long contexts with an eighth of the heads and two tokens to verify
        {"name": "decode long", "op": "decode", "batch": 32, "shortest": 64, "longest": 16384, "heads": 16, "new": 2, "dtype": "f16"},
        # one decode step of a batch of 64
        {"name": "output step", "op": "output", "tokens": 64, "heads": 128, "dtype": "bf16"},
        # a chunk of verified tokens with a quarter of the heads
        {"name": "output chunk", "op": "output", "tokens": 1499, "heads": 32, "dtype": "f16"},
        # a short conversation read back
        {"name": "gather short", "op": "gather", "batch": 3, "longest": 300, "dtype": "bf16"},
        # long conversations read back
        {"name": "gather long", "op": "gather", "batch": 32, "longest": 16384, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("query", "append", "decode", "output", "gather", "decode"))
    c = {"op": op, "dtype": rng.choice(("bf16", "f16"))}
    if op in ("query", "output"):
        c.update(tokens=_log(rng, 1, 4096), heads=rng.choice((1, 2, 5, 8, 20, 32, 64, 128)))
        c["tokens"] = min(c["tokens"], 65536 // c["heads"])
    elif op == "append":
        c.update(batch=_log(rng, 1, 128), new=_log(rng, 1, 2048), prefix=_log(rng, 1, 8192))
        c["batch"] = max(1, min(c["batch"], 16384 // c["new"], 131072 // (c["prefix"] + c["new"])))
    elif op == "gather":
        c.update(batch=_log(rng, 1, 32), longest=_log(rng, 1, 16384))
    else:
        longest, heads, new = _log(rng, 1, 65536), rng.choice((1, 3, 8, 16, 20, 32, 64, 96, 128)), rng.choice((1, 1, 1, 2, 3, 4))
        c.update(longest=longest, shortest=rng.randint(0, longest), heads=heads, new=new)
        c.update(batch=max(1, min(_log(rng, 1, 128), (1 << 19) // longest, (1 << 25) // (longest * heads * new))))
    if op in ("query", "append"):
        c.update(interleaved=rng.random() < 0.5)
    return c


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], hi among them: the same ones for the same arguments."""
    r = random.Random("%s %s %s" % (n, lo, hi))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _lengths(case):
    """Keys cached per sequence: before the pass (append), or to attend over or read."""
    if case["op"] == "decode":
        return _spread(case["batch"], case["shortest"], case["longest"])
    if case["op"] == "gather":
        return _spread(case["batch"], min(1, case["longest"]), case["longest"])
    return _spread(case["batch"], 0, case["prefix"])


def work(case):
    op = case["op"]
    if op == "query":
        n, h = case["tokens"] * case["heads"], case["heads"]
        return {"bytes": 2 * n * (NOPE + ROPE + ROW) + 2 * h * NOPE * LATENT + 4 * case["tokens"] * (ROPE + 1),
                "flops": n * (2 * NOPE * LATENT + 3 * ROPE)}
    if op == "output":
        n, h = case["tokens"] * case["heads"], case["heads"]
        return {"bytes": 2 * n * (LATENT + VALUE) + 2 * h * VALUE * LATENT, "flops": n * 2 * VALUE * LATENT}
    if op == "append":
        t = case["batch"] * case["new"]
        return {"bytes": t * (4 * ROW + 4 * ROPE), "flops": t * (4 * LATENT + 3 * ROPE)}
    keys = sum(_lengths(case))
    if op == "gather":
        return {"bytes": 4 * keys * ROW, "flops": 0}
    rows = case["batch"] * case["new"] * case["heads"]
    return {"bytes": 2 * keys * ROW + rows * (2 * ROW + 2 * LATENT + 4), "flops": 2 * keys * case["new"] * case["heads"] * (ROW + LATENT)}


# ----------------------------------------------------------------- inputs

def _offsets(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device=DEV)


def _pages(lens, g):
    """A block table of pages in random order, and the pages of the pool."""
    need = [-(-n // PAGE) for n in lens]
    width, total = max(1, max(need)), max(1, sum(need)) + 2
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    n = torch.tensor(need, device=DEV)
    first = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col).clamp(max=total - 1)
    return torch.where(col < n[:, None], order[at], torch.zeros_like(order[at])).contiguous(), total


def _make_pool(pages, dtype, g):
    """Normed latent vectors under a weight, and rotary parts of their own size."""
    gain = torch.cat((1 + 0.2 * torch.randn(LATENT, generator=g, device=DEV), 1.5 + 0.3 * torch.randn(ROPE, generator=g, device=DEV)))
    pool = torch.empty((pages, PAGE, ROW), dtype=dtype, device=DEV)
    for lo in range(0, pages, 2048):
        n = min(2048, pages - lo)
        pool[lo:lo + n] = torch.randn((n, PAGE, ROW), generator=g, device=DEV) * gain
    return pool


def _angles():
    pairs = ROPE // 2
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
    angle = torch.arange(MAX_POS, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def _up_projection(heads, dtype, g):
    """Every head's key and value up-projections in one packed weight, as they are loaded."""
    return (torch.randn((heads, NOPE + VALUE, LATENT), generator=g, device=DEV) * LATENT ** -0.5).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, dt = case["op"], T16[case["dtype"]]
    s = {"case": case}
    if op == "query":
        t, h = case["tokens"], case["heads"]
        s["q"] = torch.randn((t, h, NOPE + ROPE), generator=g, device=DEV).to(dt)
        s["w"] = _up_projection(h, dt, g)[:, :NOPE]
        s["positions"] = torch.randint(0, MAX_POS, (t,), generator=g, device=DEV, dtype=torch.int32)
        s["cos_sin"] = _angles()
        s["out"] = torch.empty((t, h, ROW), dtype=dt, device=DEV)
        if own:
            _own_query(s)
        return s
    if op == "output":
        t, h = case["tokens"], case["heads"]
        s["o"] = torch.randn((t, h, LATENT), generator=g, device=DEV).to(dt)
        s["w"] = _up_projection(h, dt, g)[:, NOPE:]
        s["out"] = torch.empty((t, h, VALUE), dtype=dt, device=DEV)
        if own:
            _own_output(s)
        return s
    lens = s["lens"] = _lengths(case)
    new = case["new"] if op == "append" else 0
    s["table"], pages = _pages([n + new for n in lens], g)
    s["pool"] = _make_pool(pages, dt, g)
    if op == "append":
        # the projection's row: latent and rotary part behind other columns
        packed = torch.randn((new * len(lens), 128 + ROW), generator=g, device=DEV).to(dt)
        s["kv"] = packed[:, 128:]
        s["weight"] = (1 + 0.2 * torch.randn(LATENT, generator=g, device=DEV)).to(dt)
        s["start"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["cu"] = _offsets([new] * len(lens))
        s["cos_sin"] = _angles()
        s["eps"] = 1e-6
        if own:
            _own_append(s)
    elif op == "gather":
        s["start"] = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
        s["cu"] = _offsets(lens)
        s["latent"] = torch.empty((sum(lens), LATENT), dtype=dt, device=DEV)
        s["rope"] = torch.empty((sum(lens), 1, ROPE), dtype=dt, device=DEV)
        if own:
            _own_gather(s)
    else:
        b, h, n = case["batch"], case["heads"], case["new"]
        s["q"] = torch.randn((b * n, h, ROW), generator=g, device=DEV).to(dt)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["out"] = torch.empty((b * n, h, LATENT), dtype=dt, device=DEV)
        s["lse"] = torch.empty((b * n, h), device=DEV)
        if own:
            _own_decode(s)
    return s


# ----------------------------------------------------------------- plain forms

def _turn(x, at, cos_sin, interleaved):
    """x fp32 [T, ..., 64] turned by the angles of the positions `at` [T]."""
    half = ROPE // 2
    rows = cos_sin[at.long()].reshape(at.shape[:1] + (1,) * (x.dim() - 2) + (ROPE,))
    cos, sin = rows[..., :half], rows[..., half:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)


def _plain_query(s, case):
    q = s["q"].float()
    absorbed = torch.matmul(q[..., :NOPE].transpose(0, 1), s["w"].float()).transpose(0, 1)
    turned = _turn(q[..., NOPE:], s["positions"], s["cos_sin"], case["interleaved"])
    return torch.cat((absorbed, turned), -1).to(s["q"].dtype)


def _plain_output(s, case):
    out = torch.matmul(s["o"].float().transpose(0, 1), s["w"].float().transpose(1, 2)).transpose(0, 1)
    return out.to(s["o"].dtype).contiguous()


def _plain_append(s, case):
    x = s["kv"].float()
    c = x[:, :LATENT]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    at = (s["start"][:, None] + torch.arange(case["new"], device=DEV)).flatten()
    b = torch.arange(s["start"].shape[0], device=DEV).repeat_interleave(case["new"])
    rows = torch.cat((c, _turn(x[:, LATENT:], at, s["cos_sin"], case["interleaved"])), -1)
    s["pool"][s["table"][b, at // PAGE].long(), at % PAGE] = rows.to(s["pool"].dtype)


def _plain_gather(s, case):
    total = s["latent"].shape[0]
    counts = s["cu"].diff()
    b = torch.repeat_interleave(torch.arange(counts.shape[0], device=DEV), counts, output_size=total)
    at = torch.arange(total, device=DEV) - s["cu"][b] + s["start"][b]
    rows = s["pool"][s["table"][b, at // PAGE].long(), at % PAGE]
    return rows[:, :LATENT].contiguous(), rows[:, None, LATENT:].contiguous()


def _plain_decode(s, case):
    b, h, n = case["batch"], case["heads"], case["new"]
    kv = s["pool"][s["table"].long()].flatten(1, 2).float()  # [B, keys, 576]
    score = torch.matmul(s["q"].float().reshape(b, n * h, ROW), kv.transpose(1, 2)) * SCALE
    sees = s["seq_lens"][:, None] - (n - 1 - torch.arange(n, device=DEV))  # [B, new]: keys that a token sees
    dead = torch.arange(kv.shape[1], device=DEV) >= sees.repeat_interleave(h, 1)[..., None]
    score = score.masked_fill(dead, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[..., :LATENT]) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    return out.to(s["q"].dtype).reshape(b * n, h, LATENT), lse.reshape(b * n, h)


# ----------------------------------------------------------------- the library's calls

def _own_query(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    from paged_kv_attention_fwd_gb300 import ops
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    sh = ops.mla_query_shapes(s["q"], s["w"], max_position=MAX_POS, interleaved=s["case"]["interleaved"], out=s["out"])
    s["call"] = B.prepared("pa_mla_query", sh, s["q"], s["w"], s["positions"], s["cos_sin"], s["out"], s["workspace"],
                           B.PA_STATUS_BYTES)


def _own_output(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    from paged_kv_attention_fwd_gb300 import ops
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    sh = ops.mla_output_shapes(s["o"], s["w"], out=s["out"])
    s["call"] = B.prepared("pa_mla_output", sh, s["o"], s["w"], s["out"], s["workspace"], B.PA_STATUS_BYTES)


def _cache_shapes(s, total, **more):
    from paged_kv_attention_fwd_gb300 import ops
    c = s["case"]
    return ops.mla_cache_shapes(c["batch"], s["table"].shape[1], s["pool"].shape[0], total, dtype=c["dtype"], **more)


def _own_append(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    sh = _cache_shapes(s, s["kv"].shape[0], kv=s["kv"], max_position=MAX_POS, interleaved=s["case"]["interleaved"], eps=s["eps"])
    s["call"] = B.prepared("pa_mla_append_kv", sh, s["kv"], s["weight"], None, s["cos_sin"], s["cu"], s["start"],
                           s["table"], s["pool"], s["workspace"], B.PA_STATUS_BYTES)


def _own_gather(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    s["call"] = B.prepared("pa_mla_gather_kv", _cache_shapes(s, s["latent"].shape[0]), s["pool"], s["cu"], s["start"],
                           s["table"], s["latent"], s["rope"], s["workspace"], B.PA_STATUS_BYTES)


def _own_decode(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    from paged_kv_attention_fwd_gb300 import ops
    c = s["case"]
    sh = ops.mla_decode_shapes(c["batch"], c["heads"], s["table"].shape[1], s["pool"].shape[0], q_len=c["new"],
                               dtype=c["dtype"], device=DEV)
    s["workspace"] = torch.zeros(B.pa_mla_decode_workspace_size(sh), dtype=torch.uint8, device=DEV)
    s["call"] = B.prepared("pa_mla_decode", sh, s["q"], s["pool"], s["table"], s["seq_lens"], SCALE, s["out"], s["lse"],
                           s["workspace"], s["workspace"].numel())


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        s["call"]()
        if op == "append":
            return {"pool": s["pool"]}
        if op == "gather":
            return {"latent": s["latent"], "rope": s["rope"]}
        return {"out": s["out"], "lse": s["lse"]} if op == "decode" else {"out": s["out"]}
    if op == "query":
        return {"out": _plain_query(s, case)}
    if op == "output":
        return {"out": _plain_output(s, case)}
    if op == "append":
        _plain_append(s, case)
        return {"pool": s["pool"]}
    if op == "gather":
        latent, rope = _plain_gather(s, case)
        return {"latent": latent, "rope": rope}
    out, lse = _plain_decode(s, case)
    return {"out": out, "lse": lse}


# ----------------------------------------------------------------- in 64 bits

def _exact_turn(x, at, cos_sin, interleaved):
    """Each pair as a complex number times the angle's."""
    half = ROPE // 2
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    w = cos_sin.double()[at.long()]
    angle = torch.complex(w[:, :half], w[:, half:])
    z = torch.complex(x[..., first].double(), x[..., second].double()) * angle.view((at.shape[0],) + (1,) * (x.dim() - 2) + (half,))
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "query":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
        for h in range(case["heads"]):
            out[:, h, :LATENT] = s["q"][:, h, :NOPE].double() @ s["w"][h].double()
        out[..., LATENT:] = _exact_turn(s["q"][..., NOPE:], s["positions"], s["cos_sin"], case["interleaved"])
        return {"out": out}
    if op == "output":
        return {"out": torch.stack([s["o"][:, h].double() @ s["w"][h].double().T for h in range(case["heads"])], 1)}
    table = s["table"].cpu()
    if op == "append":
        pool = s["pool"].double()
        x = s["kv"].double()
        c = x[:, :LATENT]
        c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / LATENT + s["eps"]) * s["weight"].double()
        at = [(b, n + i) for b, n in enumerate(s["lens"]) for i in range(case["new"])]
        rope = _exact_turn(s["kv"][:, LATENT:], torch.tensor([p for _, p in at], device=DEV), s["cos_sin"], case["interleaved"])
        page = torch.tensor([int(table[b, p // PAGE]) for b, p in at], device=DEV)
        row = torch.tensor([p % PAGE for _, p in at], device=DEV)
        pool[page, row] = torch.cat((c, rope), -1)
        return {"pool": pool}
    keys = [s["pool"][table[b, : -(-n // PAGE)].long().to(DEV)].flatten(0, 1)[:n].double() for b, n in enumerate(s["lens"])]
    if op == "gather":
        rows = torch.cat(keys)
        return {"latent": rows[:, :LATENT], "rope": rows[:, None, LATENT:]}
    new, h = case["new"], case["heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, k in enumerate(keys):
        for i in range(new):
            n = k.shape[0] - (new - 1 - i)
            if n <= 0:
                continue
            t = b * new + i
            score = (s["q"][t].double() @ k[:n].T) / math.sqrt(NOPE + ROPE)
            lse[t] = torch.logsumexp(score, -1)
            out[t] = torch.exp(score - lse[t, :, None]) @ k[:n, :LATENT]
    return {"out": out, "lse": lse}
