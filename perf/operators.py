"""Cases of the serving step around a 4-bit paged KV cache.

Five operators, each in its plain form (elementary torch operations in fp32)
and, where `own` is set, as the calls a user makes of the library:

  norm_rope    RMS norm of every query and key head, then the rotary position
               rotation (one or several position axes), in one pass
  step_append  the same, with the keys and values going straight into their
               cache pages
  cache4       quantising new keys and values into 4-bit pages as they are
               written, and reading a sequence's rows back
  read_back    reading rows of a paged cache (4-bit, e4m3 or 16-bit pages) back
               as the ragged 16-bit tensors a prefill takes
  decode4      single-token attention over the 4-bit cache

The 4-bit page slab of one KV head is 64 rows of D/2 bytes (e2m1 codes, element
2i in the low nibble of byte i) followed by 64 rows of D/16 bytes (one e4m3
scale per 16 elements).  An element stands for code * block scale * head scale.
"""
import math
import random

import torch

own = False

PAGE = 64
DEV = "cuda"
MAX_POS = 32768
# e2m1 magnitudes by code
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
T16 = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence: the latency of a decode step's first kernel
        {"name": "norm_rope token", "op": "norm_rope", "tokens": 1, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "axes": 1, "interleaved": False, "dtype": "bf16"},
        # an image / video prompt: three position axes, part of the head rotated, an odd token count
        {"name": "norm_rope video", "op": "norm_rope", "tokens": 4097, "hq": 16, "hk": 4, "d": 64, "rot": 48,
         "axes": 3, "interleaved": True, "dtype": "f16"},
        # a long prompt out of a packed qkv projection
        {"name": "norm_rope prompt", "op": "norm_rope", "tokens": 16384, "hq": 64, "hk": 8, "d": 128, "rot": 128,
         "axes": 1, "interleaved": False, "dtype": "bf16"},
        # one decode step of a batch of 64
        {"name": "step_append step", "op": "step_append", "batch": 64, "new": 1, "prefix": 4096, "hq": 32, "hk": 8,
         "d": 128, "rot": 128, "axes": 1, "interleaved": False, "dtype": "bf16"},
        # chunks of eight prompts
        {"name": "step_append chunk", "op": "step_append", "batch": 8, "new": 512, "prefix": 8192, "hq": 32, "hk": 8,
         "d": 128, "rot": 128, "axes": 1, "interleaved": False, "dtype": "bf16"},
        # one decode step of a batch of 64 into the 4-bit cache
        {"name": "cache4 step", "op": "cache4", "batch": 64, "new": 1, "prefix": 4096, "hk": 8, "d": 128, "whole": False},
        # chunks of eight prompts written, and all that each sequence has cached read back for the prefill
        {"name": "cache4 chunk", "op": "cache4", "batch": 8, "new": 512, "prefix": 8192, "hk": 8, "d": 128, "whole": True},
        # a short conversation read back
        {"name": "read_back short", "op": "read_back", "batch": 3, "longest": 300, "hk": 8, "d": 128, "kv": "fp4"},
        # long conversations read back
        {"name": "read_back long", "op": "read_back", "batch": 32, "longest": 16384, "hk": 8, "d": 128, "kv": "fp4"},
        # one short sequence: the latency of an attention call
        {"name": "decode4 one", "op": "decode4", "batch": 1, "shortest": 777, "longest": 777, "hq": 32, "hk": 8, "d": 128},
        # the GQA decode batch: 64 sequences of 1 to 4096 keys
        {"name": "decode4 batch", "op": "decode4", "batch": 64, "shortest": 1, "longest": 4096, "hq": 32, "hk": 8, "d": 128},
        # the long-context batch: 128 sequences of up to 8192 keys, eight query heads to a KV head
        {"name": "decode4 long", "op": "decode4", "batch": 128, "shortest": 64, "longest": 8192, "hq": 64, "hk": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "step_append", "cache4", "read_back", "decode4"))
    hk = rng.choice((1, 2, 3, 4, 5, 8))
    d = rng.choice((64, 128))
    c = {"op": op, "hk": hk, "d": d}
    if op in ("norm_rope", "step_append"):
        c.update(hq=hk * rng.choice((1, 2, 4, 5, 8)), rot=8 * rng.randint(1, d // 8), axes=rng.choice((1, 1, 2, 3)),
                 interleaved=rng.random() < 0.5, dtype=rng.choice(("bf16", "f16")))
    if op == "norm_rope":
        c.update(tokens=_log(rng, 1, 16384))
    elif op in ("step_append", "cache4"):
        c.update(batch=_log(rng, 1, 64), new=_log(rng, 1, 512), prefix=_log(rng, 1, 8192))
        c["batch"] = max(1, min(c["batch"], 4096 // c["new"], 131072 // (c["prefix"] + c["new"])))
        if op == "cache4":
            c.update(whole=rng.random() < 0.5)
    elif op == "read_back":
        c.update(batch=_log(rng, 1, 32), longest=_log(rng, 1, 16384), kv=rng.choice(("fp4", "fp4", "e4m3", "bf16", "f16")))
    else:
        longest = _log(rng, 1, 65536)
        c.update(hq=hk * rng.choice((1, 2, 4, 6, 8, 16)), longest=longest, shortest=rng.randint(0, longest))
        c.update(batch=max(1, min(_log(rng, 1, 256), 262144 // longest)))
    return c


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], hi among them: the same ones for the same arguments."""
    r = random.Random("%s %s %s" % (n, lo, hi))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _lengths(case):
    """Keys cached per sequence before the pass."""
    if case["op"] == "decode4":
        return _spread(case["batch"], case["shortest"], case["longest"])
    if case["op"] == "read_back":
        return _spread(case["batch"], min(1, case["longest"]), case["longest"])
    return _spread(case["batch"], 0, case["prefix"])


def _slab(d, kv):
    return PAGE * {"fp4": d // 2 + d // 16, "e4m3": d}.get(kv, 2 * d)


def work(case):
    d, hk, op = case["d"], case["hk"], case["op"]
    if op == "norm_rope":
        t, h = case["tokens"], case["hq"] + hk
        return {"bytes": 4 * t * h * d + t * (4 * case["rot"] + 4 * case["axes"]), "flops": t * h * (4 * d + 3 * case["rot"])}
    if op == "step_append":
        t, h = case["batch"] * case["new"], case["hq"] + 2 * hk
        return {"bytes": 4 * t * h * d + t * (4 * case["rot"] + 4 * case["axes"]), "flops": t * (h - hk) * (4 * d + 3 * case["rot"])}
    if op == "cache4":
        new, row = case["batch"] * case["new"], 2 * hk * d
        read = new + sum(_lengths(case)) if case["whole"] else new
        # new rows in 16 bits in and 4.5 bits out; rows in 4.5 bits in and 16 bits out
        return {"bytes": new * row * (2 + 0.5625) + read * row * (0.5625 + 2), "flops": new * row * 3 + read * row * 2}
    if op == "read_back":
        read = sum(_lengths(case))
        return {"bytes": 2 * hk * read * (_slab(d, case["kv"]) / PAGE + 2 * d), "flops": 2 * hk * read * d * 2}
    keys = sum(_lengths(case))
    rows = case["batch"] * case["hq"]
    return {"bytes": 2 * hk * keys * (d // 2 + d // 16) + rows * (4 * d + 4), "flops": 4 * keys * case["hq"] * d}


# ----------------------------------------------------------------- 4 bits, plainly

def _to_fp4(x, head):
    """x fp32 [..., D] and the head scale [..., 1] -> codes uint8 [..., D] and block scales e4m3 [..., D/16]."""
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    scale = (amax / (head * 6)).clamp(max=448).to(torch.float8_e4m3fn)
    step = (scale.float() * head).unsqueeze(-1)
    t = torch.where(step > 0, blocks.abs() / step, torch.zeros_like(blocks)).clamp(max=6)
    v = torch.where(t < 2, (t * 2).round() / 2, torch.where(t < 4, t.round(), (t / 2).round() * 2))
    code = torch.where(v < 2, v * 2, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    code = torch.where(step > 0, code + 8 * torch.signbit(blocks).to(torch.uint8), torch.zeros_like(code))
    return code.flatten(-2), scale


def _fp4_rows(x, head):
    """x fp32 [..., D] -> code bytes [..., D/2] and scale bytes [..., D/16]."""
    code, scale = _to_fp4(x, head)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8)


def _byte_pairs(dtype):
    """[256, 2]: the two e2m1 values of a byte, the low nibble's first."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=dtype, device=DEV)
    b = torch.arange(256, device=DEV)
    return torch.stack((grid[b & 15], grid[b >> 4]), -1)


def _from_fp4(byte_pairs, codes, scales, head):
    """Code bytes [..., D/2], scale bytes [..., D/16], head scale [..., 1] -> fp32 [..., D]."""
    v = byte_pairs[codes.long()].flatten(-2).unflatten(-1, (-1, 16))
    return (v * (scales.view(torch.float8_e4m3fn).float() * head).unsqueeze(-1)).flatten(-2)


def _pool_rows(byte_pairs, pool, page, row, d, kv, head):
    """Rows `row` of the pages `page` (same shapes [N]) of every head: fp32 [N, Hk, D]."""
    if kv == "fp4":
        codes = pool[..., : PAGE * d // 2].unflatten(-1, (PAGE, d // 2))[page, :, row]
        scales = pool[..., PAGE * d // 2:].unflatten(-1, (PAGE, d // 16))[page, :, row]
        return _from_fp4(byte_pairs, codes, scales, head.view(-1, 1))
    x = pool[page, :, row].float()
    return x * head.view(-1, 1) if kv == "e4m3" else x


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


def _heads_of(x_gain, shape, g, dtype):
    """Keys or values as a projection leaves them: normal, with channels of unequal size."""
    return (torch.randn(shape, generator=g, device=DEV) * x_gain).to(dtype)


def _make_pool(pages, hk, d, kv, g):
    """A filled pool and its head scales (of ones where the type has none)."""
    gain = torch.exp(0.5 * torch.randn((hk, 1, d), generator=g, device=DEV))
    if kv in T16:
        return _heads_of(gain, (pages, hk, PAGE, d), g, T16[kv]), torch.ones(hk, device=DEV)
    top = gain.amax((1, 2)) * 5
    if kv == "e4m3":
        head = top / 448
        x = torch.randn((pages, hk, PAGE, d), generator=g, device=DEV) * gain / head.view(-1, 1, 1)
        return x.clamp(-448, 448).to(torch.float8_e4m3fn), head
    head = top / (6 * 448)
    pool = torch.empty((pages, hk, _slab(d, kv)), dtype=torch.uint8, device=DEV)
    for lo in range(0, pages, 4096):
        n = min(4096, pages - lo)
        codes, scales = _fp4_rows(_heads_of(gain, (n, hk, PAGE, d), g, torch.bfloat16).float(), head.view(-1, 1, 1))
        pool[lo:lo + n, :, : PAGE * d // 2] = codes.flatten(-2)
        pool[lo:lo + n, :, PAGE * d // 2:] = scales.flatten(-2)
    return pool, head


def _rope_inputs(case, tokens, positions, g):
    """What norm_rope and step_append share: packed projections, weights, positions, the angle table."""
    hq, hk, d, rot = case["hq"], case["hk"], case["d"], case["rot"]
    dt = T16[case["dtype"]]
    qkv = torch.randn((tokens, (hq + 2 * hk) * d), generator=g, device=DEV).to(dt)
    pairs = rot // 2
    freq = 1e6 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
    angle = torch.arange(MAX_POS, dtype=torch.float64, device=DEV)[:, None] * freq
    sections = [pairs // case["axes"]] * case["axes"]
    sections[0] += pairs - sum(sections)
    return {
        "q": qkv[:, : hq * d].unflatten(-1, (hq, d)), "k": qkv[:, hq * d:(hq + hk) * d].unflatten(-1, (hk, d)),
        "v": qkv[:, (hq + hk) * d:].unflatten(-1, (hk, d)),
        "q_weight": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt),
        "k_weight": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt),
        "positions": positions, "cos_sin": torch.cat((angle.cos(), angle.sin()), -1).float(),
        "sections": sections, "eps": 1e-6,
        "axis": torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=DEV), "q_out": torch.empty((tokens, hq, d), dtype=dt, device=DEV),
    }


def _token_places(s, new):
    """Page and row of each sequence's `new` tokens after those it has cached, in order."""
    pos = (s["start"][:, None] + torch.arange(new, device=DEV)).flatten()
    b = torch.arange(s["start"].shape[0], device=DEV).repeat_interleave(new)
    return s["table"][b, pos // PAGE].long(), pos % PAGE


def _row_places(s):
    """Page and row of the rows that each sequence in turn reads back."""
    total = s["k_rows"].shape[0]
    counts = s["cu_read"].diff()
    b = torch.repeat_interleave(torch.arange(counts.shape[0], device=DEV), counts, output_size=total)
    pos = torch.arange(total, device=DEV) - s["cu_read"][b] + s["first_dev"][b]
    return s["table"][b, pos // PAGE].long(), pos % PAGE


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, hk, d = case["op"], case["hk"], case["d"]
    s = {"case": case, "byte_pairs": _byte_pairs(torch.float32)}
    if op == "norm_rope":
        t = case["tokens"]
        # positions of every axis: a run of tokens in time, random places in height and width
        at = torch.randint(0, MAX_POS - t, (1,), generator=g, device=DEV) + torch.arange(t, device=DEV)
        pos = torch.stack([at] + [torch.randint(0, 64, (t,), generator=g, device=DEV) for _ in range(case["axes"] - 1)])
        s.update(_rope_inputs(case, t, pos.to(torch.int32).contiguous(), g))
        s["k_out"] = torch.empty((t, hk, d), dtype=s["q_out"].dtype, device=DEV)
        if own:
            _own_norm_rope(s)
        return s
    lens = _lengths(case)
    s["lens"] = lens
    if op in ("step_append", "cache4"):
        new = case["new"]
        total = [n + new for n in lens]
        kv = case["dtype"] if op == "step_append" else "fp4"
        s["table"], pages = _pages(total, g)
        s["k_pool"], s["k_scale"] = _make_pool(pages, hk, d, kv, g)
        s["v_pool"], s["v_scale"] = _make_pool(pages, hk, d, kv, g)
        s["start"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["cu_new"] = _offsets([new] * len(lens))
        if op == "step_append":
            pos = (s["start"][:, None] + torch.arange(new, dtype=torch.int32, device=DEV)).flatten()
            s.update(_rope_inputs(case, new * len(lens), pos.expand(case["axes"], -1).contiguous(), g))
            if own:
                _own_step_append(s)
            return s
        gain = torch.exp(0.5 * torch.randn((hk, d), generator=g, device=DEV))
        s["k_new"] = _heads_of(gain, (new * len(lens), hk, d), g, torch.bfloat16)
        s["v_new"] = _heads_of(gain, (new * len(lens), hk, d), g, torch.bfloat16)
        s["first"], s["count"] = ([0] * len(lens), total) if case["whole"] else (lens, [new] * len(lens))
    elif op == "read_back":
        s["table"], pages = _pages(lens, g)
        s["k_pool"], s["k_scale"] = _make_pool(pages, hk, d, case["kv"], g)
        s["v_pool"], s["v_scale"] = _make_pool(pages, hk, d, case["kv"], g)
        s["first"], s["count"] = [0] * len(lens), lens
    else:
        s["table"], pages = _pages(lens, g)
        s["k_pool"], s["k_scale"] = _make_pool(pages, hk, d, "fp4", g)
        s["v_pool"], s["v_scale"] = _make_pool(pages, hk, d, "fp4", g)
        s["q"] = (1.5 * torch.randn((case["batch"], case["hq"], d), generator=g, device=DEV)).to(torch.bfloat16)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["batch"], case["hq"]), device=DEV)
        if own:
            _own_decode(s)
        return s
    s["cu_read"] = _offsets(s["count"])
    s["first_dev"] = torch.tensor(s["first"], dtype=torch.int32, device=DEV)
    dt = T16.get(case.get("kv"), torch.bfloat16)
    s["k_rows"] = torch.empty((sum(s["count"]), hk, d), dtype=dt, device=DEV)
    s["v_rows"] = torch.empty((sum(s["count"]), hk, d), dtype=dt, device=DEV)
    if own:
        _own_cache(s)
    return s


# ----------------------------------------------------------------- plain forms

def _norm_rope(x, weight, s, case, out_dtype):
    """x [T, H, D]: RMS norm over D, weight, rotation of the first `rot` elements."""
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot = case["rot"]
    pairs = rot // 2
    pair = torch.arange(pairs, device=DEV)
    at = s["positions"].long()[s["axis"]].T  # [T, pairs]
    cos, sin = s["cos_sin"][at, pair].unsqueeze(1), s["cos_sin"][at, pairs + pair].unsqueeze(1)
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"] else (y[..., :pairs], y[..., pairs:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(out_dtype)


def _plain_cache4(s, case):
    d = case["d"]
    page, row = _token_places(s, case["new"])
    for pool, new, head in ((s["k_pool"], s["k_new"], s["k_scale"]), (s["v_pool"], s["v_new"], s["v_scale"])):
        codes, scales = _fp4_rows(new.float(), head.view(-1, 1))
        pool[..., : PAGE * d // 2].unflatten(-1, (PAGE, d // 2))[page, :, row] = codes
        pool[..., PAGE * d // 2:].unflatten(-1, (PAGE, d // 16))[page, :, row] = scales


def _plain_read(s, case):
    page, row = _row_places(s)
    kv = case.get("kv", "fp4")
    dt = s["k_rows"].dtype
    return (_pool_rows(s["byte_pairs"], s["k_pool"], page, row, case["d"], kv, s["k_scale"]).to(dt),
            _pool_rows(s["byte_pairs"], s["v_pool"], page, row, case["d"], kv, s["v_scale"]).to(dt))


def _plain_decode(s, case):
    hk, d = case["hk"], case["d"]
    b, hq = case["batch"], case["hq"]
    width = s["table"].shape[1]

    def paged(pool, head):  # [B, Hk, width * 64, D]
        slab = pool[s["table"].long()]
        codes = slab[..., : PAGE * d // 2].unflatten(-1, (PAGE, d // 2))
        scales = slab[..., PAGE * d // 2:].unflatten(-1, (PAGE, d // 16))
        return _from_fp4(s["byte_pairs"], codes, scales, head.view(-1, 1, 1)).transpose(1, 2).flatten(2, 3)

    q = s["q"].float().unflatten(1, (hk, hq // hk))
    score = torch.matmul(q, paged(s["k_pool"], s["k_scale"]).transpose(-1, -2)) * d ** -0.5
    dead = torch.arange(width * PAGE, device=DEV) >= s["seq_lens"][:, None]
    score = score.masked_fill(dead[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, paged(s["v_pool"], s["v_scale"])) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    return out.reshape(b, hq, d).to(torch.bfloat16), lse.reshape(b, hq)


# ----------------------------------------------------------------- the library's calls

def _rope_shapes(s):
    from paged_kv_attention_fwd_gb300 import ops
    c = s["case"]
    return ops.rope_shapes(s["q"], s["k"], v=s["v"], rope_dim=c["rot"], max_position=MAX_POS, interleaved=c["interleaved"],
                           sections=s["sections"], eps=s["eps"])


def _own_norm_rope(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    s["call"] = B.prepared("pa_qk_norm_rope", _rope_shapes(s), s["q"], s["k"], s["q_weight"], s["k_weight"],
                           s["positions"], s["cos_sin"], s["q_out"], s["k_out"], s["workspace"], B.PA_STATUS_BYTES)


def _append_shapes(s, total, kv):
    from paged_kv_attention_fwd_gb300 import binding as B
    c = s["case"]
    return B.pa_append_shapes(batch=c["batch"], num_kv_heads=c["hk"], head_dim=c["d"], page_size=PAGE,
                              max_pages_per_seq=s["table"].shape[1], num_pool_pages=s["k_pool"].shape[0], total_new=total,
                              kv_dtype={"bf16": B.PA_KV_BF16, "f16": B.PA_KV_FP16, "e4m3": B.PA_KV_FP8_E4M3,
                                        "fp4": B.PA_KV_FP4_E2M1}[kv])


def _own_step_append(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    c = s["case"]
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    s["call"] = B.prepared("pa_norm_rope_append_kv", _rope_shapes(s), _append_shapes(s, s["q"].shape[0], c["dtype"]),
                           s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["cos_sin"],
                           s["cu_new"], s["start"], s["table"], s["q_out"], s["k_pool"], s["v_pool"], None, None,
                           s["workspace"], B.PA_STATUS_BYTES)


def _own_cache(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    kv = s["case"].get("kv", "fp4")
    scales = (None, None) if kv in T16 else (s["k_scale"], s["v_scale"])
    s["workspace"] = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    if "k_new" in s:
        s["write"] = B.prepared("pa_append_kv", _append_shapes(s, s["k_new"].shape[0], kv), s["k_new"], s["v_new"],
                                s["cu_new"], s["start"], s["table"], s["k_pool"], s["v_pool"], *scales, s["workspace"],
                                B.PA_STATUS_BYTES)
    s["read"] = B.prepared("pa_gather_kv", _append_shapes(s, s["k_rows"].shape[0], kv), s["k_pool"], s["v_pool"], *scales,
                           s["cu_read"], s["first_dev"], s["table"], s["k_rows"], s["v_rows"], s["workspace"],
                           B.PA_STATUS_BYTES)


def _own_decode(s):
    from paged_kv_attention_fwd_gb300 import binding as B
    from paged_kv_attention_fwd_gb300 import ops
    c = s["case"]
    p = s["plan"] = ops.plan_decode(s["lens"], None, c["hq"], c["hk"], c["d"], s["table"].shape[1], s["k_pool"].shape[0],
                                    kv_dtype="fp4", device=DEV)
    s["call"] = B.prepared("pa_decode", p.shapes, p.plan, s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                           s["table"], s["seq_lens"], p.meta_dev, c["d"] ** -0.5, s["out"], s["lse"], p.workspace,
                           p.workspace.numel())


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_rope":
        if own:
            s["call"]()
            return {"q": s["q_out"], "k": s["k_out"]}
        return {"q": _norm_rope(s["q"], s["q_weight"], s, case, s["q"].dtype),
                "k": _norm_rope(s["k"], s["k_weight"], s, case, s["k"].dtype)}
    if op == "step_append":
        if own:
            s["call"]()
            q = s["q_out"]
        else:
            q = _norm_rope(s["q"], s["q_weight"], s, case, s["q"].dtype)
            page, row = _token_places(s, case["new"])
            s["k_pool"][page, :, row] = _norm_rope(s["k"], s["k_weight"], s, case, s["k"].dtype)
            s["v_pool"][page, :, row] = s["v"]
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op in ("cache4", "read_back"):
        if own:
            if op == "cache4":
                s["write"]()
            s["read"]()
            return {"k": s["k_rows"], "v": s["v_rows"]}
        if op == "cache4":
            _plain_cache4(s, case)
        k, v = _plain_read(s, case)
        return {"k": k, "v": v}
    if own:
        s["call"]()
        return {"out": s["out"], "lse": s["lse"]}
    out, lse = _plain_decode(s, case)
    return {"out": out, "lse": lse}


# ----------------------------------------------------------------- in 64 bits

def _exact_turn(x, weight, s, case):
    x = x.double()
    y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * weight.double()
    rot, half = case["rot"], case["rot"] // 2
    z = y.clone()
    p = 0
    for axis, n in enumerate(s["sections"]):
        for pair in range(p, p + n):
            i, j = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
            rows = s["cos_sin"][s["positions"][axis].long()].double()
            c, w = rows[:, None, pair], rows[:, None, half + pair]
            z[..., i] = y[..., i] * c - y[..., j] * w
            z[..., j] = y[..., i] * w + y[..., j] * c
        p += n
    return z


def _exact_fp4(x, head):
    """The value each element of x [..., D] is stored as: nearest grid value, ties to the even code."""
    b = x.unflatten(-1, (-1, 16))
    h = head.float().reshape(-1, 1)
    scale = (b.float().abs().amax(-1) / (h * 6)).clamp(max=448).to(torch.float8_e4m3fn).float()
    step = (scale * h).unsqueeze(-1)
    t = (b.float().abs() / step).double()  # the quotient is an fp32 one by definition
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    best = torch.zeros_like(t)
    for i in range(1, 8):
        mid = (grid[i - 1] + grid[i]) / 2
        best = torch.where((t > mid) | ((t == mid) & (i % 2 == 0)), grid[i], best)
    v = torch.where(step > 0, best, torch.zeros_like(best)) * torch.sign(b.double())
    return (v * scale.double().unsqueeze(-1) * h.double().unsqueeze(-1)).flatten(-2)


def _exact_slab_rows(slab, d, kv, head):
    """One head's rows of whole pages [n, slab] -> float64 [n * 64, D]."""
    if kv in T16:
        return slab.double().flatten(0, 1)
    if kv == "e4m3":
        return slab.double().flatten(0, 1) * head.double()
    grid = torch.tensor(GRID, dtype=torch.float64, device=slab.device)
    b = slab[:, : PAGE * d // 2].reshape(-1, d // 2).int()
    n = torch.stack((b % 16, b // 16), -1).flatten(-2)
    v = torch.where(n >= 8, -grid[n % 8], grid[n % 8])
    sc = slab[:, PAGE * d // 2:].reshape(-1, d // 16).contiguous().view(torch.float8_e4m3fn).double()
    return v * sc.repeat_interleave(16, -1) * head.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, d, hk = case["op"], case["d"], case["hk"]
    if op in ("norm_rope", "step_append"):
        q, k = _exact_turn(s["q"], s["q_weight"], s, case), _exact_turn(s["k"], s["k_weight"], s, case)
        if op == "norm_rope":
            return {"q": q, "k": k}
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        table, at = s["table"].tolist(), []
        for b, n in enumerate(s["lens"]):
            at += [(table[b][i // PAGE], i % PAGE) for i in range(n, n + case["new"])]
        page, row = torch.tensor(at, device=DEV).T
        kp[page, :, row], vp[page, :, row] = k, s["v"].double()
        return {"q": q, "k_pool": kp, "v_pool": vp}
    table = s["table"].cpu()
    if op in ("cache4", "read_back"):
        got = {}
        for name in ("k", "v"):
            head, rows = s[name + "_scale"], []
            new = _exact_fp4(s[name + "_new"], head) if op == "cache4" else None
            for b, (first, count) in enumerate(zip(s["first"], s["count"])):
                pages = table[b, : -(-(first + count) // PAGE)].long().to(DEV)
                x = torch.stack([_exact_slab_rows(s[name + "_pool"][pages, h], d, case.get("kv", "fp4"), head[h])
                                 for h in range(hk)], 1)
                if new is not None:
                    n, m = s["lens"][b], case["new"]
                    x[n:n + m] = new[b * m:(b + 1) * m]
                rows.append(x[first:first + count])
            got[name] = torch.cat(rows)
        return got
    group = case["hq"] // hk
    out = torch.zeros((case["batch"], case["hq"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["batch"], case["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"]):
        if not n:
            continue
        pages = table[b, : -(-n // PAGE)].long().to(DEV)
        for h in range(hk):
            k = _exact_slab_rows(s["k_pool"][pages, h], d, "fp4", s["k_scale"][h])[:n]
            v = _exact_slab_rows(s["v_pool"][pages, h], d, "fp4", s["v_scale"][h])[:n]
            at = slice(h * group, (h + 1) * group)
            score = (s["q"][b, at].double() @ k.T) / math.sqrt(d)
            lse[b, at] = torch.logsumexp(score, -1)
            out[b, at] = torch.exp(score - lse[b, at, None]) @ v
    return {"out": out, "lse": lse}
