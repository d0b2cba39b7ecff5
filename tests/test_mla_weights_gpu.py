"""Softmax weights of the latent decode where they can go wrong: keys whose
scores are -inf, page after page and for some heads only; fp16 weights far
below a dominant key's; long sequences whose every page shows in the output.
All against fp64 on the GPU."""
import math

import pytest
import torch

from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops

from .test_mla_gpu import DEV, HALF, SCALE, T16, TINY, Cache, decode, gen, gpu, normal, rows_at  # noqa: F401

pytestmark = pytest.mark.gpu

# Half the least step of a weight, relative to the largest weight: fp16's 2^-25, of weights held 2^7 times larger
LEAST = {"bf16": 0.0, "f16": 2.0 ** -32}


def check(c, q, scale, out, lse, seen, terms=576, depth=None, skip=()):
    """One token a sequence.  seen[b]: [heads, keys], which keys have a score above -inf; terms: products of a score that
    are not zero; depth: additions that a key's share goes through (all keys of a sequence at most)."""
    for b, n in enumerate(c.lens):
        if b in skip:
            continue
        k, live = c.rows(b), seen[b]
        k = torch.where(torch.isfinite(k), k, 0.0)
        v = k[:, :512]
        s = torch.where(live, q[b].double() @ k.T * scale, -math.inf)
        none = ~live.any(-1)
        assert (out[b, none] == 0).all() and (lse[b, none] == -math.inf).all(), b
        reach = torch.where(live, q[b].double().abs() @ k.abs().T * abs(scale), 0.0).amax(-1)
        want = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(none, 0.0, want)[:, None])
        o, spread = p @ v, p @ v.abs()
        # a score: its fp32 products and the steps up to the exponent (2^-23 of its reach each), the exponential 2^-21;
        # fp32 sums of values and of weights, 2^-23 an addition (truncation included)
        sums = min(n, depth or n) * 2.0 ** -23
        logit = (terms + 4) * 2.0 ** -23 * reach + 2.0 ** -21
        rounded = torch.maximum(HALF[c.dtype] * p, LEAST[c.dtype] * p.amax(-1, keepdim=True)) * live
        tol = HALF[c.dtype] * o.abs() + rounded @ v.abs() + (2 * logit[:, None] + 2 * sums) * spread + TINY[c.dtype]
        assert torch.isfinite(out[b]).all()
        off = (out[b].double() - o).abs()
        assert (off <= tol).all(), (b, (off / tol).max().item(), (off / tol).amax(-1).argmax().item())
        ltol = logit + sums + 2.0 ** -22 * (want.abs() + 1)
        off = (lse[b].double() - want).abs()
        assert (off[~none] <= ltol[~none]).all(), (b, (off / ltol)[~none].max().item())


# ----------------------------------------------------------------- scores of -inf

LAYOUTS = {  # lengths, SMs
    "whole": ([700, 100, 320], 1),      # one range: no sequence is split
    "few": ([3000], None),              # a sequence over many SMs
    "many": ([700, 64, 333] * 10, 60),  # split, and too many sequences for the other merge
}


def hidden_case(layout, heads, first, dtype, every, rising, value):
    lens, sms = LAYOUTS[layout]
    c = Cache(lens, dtype, seed=max(first, 0))
    q = normal((len(lens), heads, 576), 1, dtype)
    hides = torch.arange(heads, device=DEV) % every == 0
    q[:, :, 575] = torch.where(hides, 4.0, 0.0).to(T16[dtype])
    seen = []
    for b, n in enumerate(lens):
        at = rows_at(c.table, b, 0, n)
        gone = torch.arange(n, device=DEV) < (n - 70 if first < 0 else first)
        c.pool.view(-1, 576)[at, 575] = torch.where(gone, value, 0.0).to(T16[dtype])
        if rising:
            c.pool.view(-1, 576)[at, 574] = (torch.arange(n, device=DEV) // 50).to(T16[dtype])
        seen.append(~(gone & hides[:, None]))
    if rising:  # 2^1.5 every 50 keys: some columns' references change now and again
        q[:, :, 574] = torch.where(torch.arange(heads, device=DEV) % 5 < 2, 14.0, 0.0).to(T16[dtype])
    return c, q, seen, sms


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("first", [64, 128, 130, -1])
@pytest.mark.parametrize("heads", [5, 32, 64, 100])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_prefix_hidden_from_some_heads(layout, heads, first, rising):
    """The first keys (-1: all but 70) at bf16's lowest value in one element, times 4: a product of -inf."""
    c, q, seen, sms = hidden_case(layout, heads, first, "bf16", 3, rising, torch.finfo(torch.bfloat16).min)
    check(c, q, SCALE, *decode(c, q, sms=sms), seen)


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("first", [64, 130, -1, 10000])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_prefix_hidden_from_all_heads(dtype, layout, first, rising):
    """Keys of -inf; with 10000 no key of any sequence is left."""
    c, q, seen, sms = hidden_case(layout, 16, first, dtype, 1, rising, -math.inf)
    check(c, q, SCALE, *decode(c, q, sms=sms), seen)


@pytest.mark.parametrize("later", [-200.0, -3.0, 0.0, 5.0, 40.0])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_scores_behind_a_hidden_prefix(layout, later):
    """Far below 1, near it and above it, in units of e."""
    lens, sms = LAYOUTS[layout]
    c = Cache(lens, "bf16", seed=2)
    q = normal((len(lens), 20, 576), 1)
    q[:, :, 575], q[:, :, 574] = 4.0, 1.0
    seen = []
    for b, n in enumerate(lens):
        at = rows_at(c.table, b, 0, n)
        gone = torch.arange(n, device=DEV) < min(200, n - 1)
        c.pool.view(-1, 576)[at, 575] = torch.where(gone, -math.inf, 0.0).bfloat16()
        c.pool.view(-1, 576)[at, 574] = later / SCALE
        seen.append((~gone).expand(20, -1))
    check(c, q, SCALE, *decode(c, q, sms=sms), seen)


@pytest.mark.parametrize("first", [64, 130, -1])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_prefix_at_the_lowest_finite_value(layout, first):
    """Times 0.5: scores of -1.2e37, finite references that later pages leave far below.  Where they are all that a head has,
    they are all the same, in 64 bits too (what differs, 100 at most, is far below half a step), and weigh the same."""
    c, q, seen, sms = hidden_case(layout, 20, first, "bf16", 2, True, torch.finfo(torch.bfloat16).min)
    q[:, :, 575] *= 0.125
    out, lse = decode(c, q, sms=sms)
    same = [b for b, n in enumerate(c.lens) if n <= first]
    check(c, q, SCALE, out, lse, seen, skip=same)
    for b in same:
        n, v, heads = c.lens[b], c.rows(b)[:, :512], ~seen[b].any(-1)
        mean, spread = v.mean(0), v.abs().mean(0)
        off = (out[b, heads].double() - mean).abs()
        assert (off <= HALF["bf16"] * mean.abs() + 2 * n * 2.0 ** -23 * spread + TINY["bf16"]).all(), b
        want = 0.5 * torch.finfo(torch.bfloat16).min * SCALE
        assert ((lse[b, heads].double() / want - 1).abs() <= 2.0 ** -20).all(), b


@pytest.mark.parametrize("q_len", [2, 4])
def test_a_hidden_prefix_and_several_tokens(q_len):
    """Hidden keys and those that a token does not see yet: each token as it is alone over its own keys."""
    lens, heads = [500, 131, 70, 64 + q_len], 16
    c = Cache(lens, "bf16", seed=3)
    q = normal((len(lens) * q_len, heads, 576), 1)
    q[:, :, 575] = 4.0
    for b, n in enumerate(lens):
        c.pool.view(-1, 576)[rows_at(c.table, b, 0, n), 575] = torch.where(torch.arange(n, device=DEV) < 64, -math.inf, 0.0).bfloat16()
    out, lse = decode(c, q, q_len)
    for i in range(q_len):
        c.lens = [n - (q_len - 1 - i) for n in lens]
        at = torch.arange(len(lens), device=DEV) * q_len + i
        seen = [(torch.arange(n, device=DEV) >= 64).expand(heads, -1) for n in c.lens]
        check(c, q[at], SCALE, out[at], lse[at], seen)


@pytest.mark.parametrize("size", [3.0, 1e3, 1e4, 3e5, 1e9, 1e37])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_equal_scores_of_any_size(dtype, layout, sign, size):
    """All keys of a sequence have the same score: they weigh the same, whatever it is and in whichever page they lie."""
    lens, sms = LAYOUTS[layout]
    c = Cache(lens, dtype, seed=8)
    top = 6e4 if dtype == "f16" else 1e38
    q = torch.zeros((len(lens), 20, 576), dtype=T16[dtype], device=DEV)
    q[..., 512] = torch.linspace(0.7, 1.0, 20, device=DEV) * min(size, 100.0)
    for b, n in enumerate(lens):
        at = rows_at(c.table, b, 0, n)
        x = c.rows(b).float()
        x[:, :512] += (torch.arange(n, device=DEV) // 64)[:, None] * 0.25  # pages apart from one another
        x[:, 512:] = 0.0
        x[:, 512] = sign * min(size / min(size, 100.0), top)
        c.pool.view(-1, 576)[at] = x.to(T16[dtype])
    out, lse = decode(c, q, scale=1.0, sms=sms)
    for b, n in enumerate(lens):
        k = c.rows(b)
        v, s = k[:, :512], q[b, :, 512].double() * k[0, 512]
        mean, spread = v.mean(0), v.abs().mean(0)
        # a weight: its rounding, and that of a score with the scale, 2^-11 at most; fp32 sums
        tol = HALF[dtype] * mean.abs() + (HALF[dtype] + 2.0 ** -10 + 2 * n * 2.0 ** -23) * spread
        off = (out[b].double() - mean).abs()
        assert (off <= tol).all(), (b, (off / tol).max().item())
        want = s + math.log(n)
        assert ((lse[b].double() - want).abs() <= 2.0 ** -21 * want.abs() + 2.0 ** -10).all(), b


# ----------------------------------------------------------------- light weights

def sink_case(n, step, sink_value, dtype, heads=16, at=317):
    """One key at score 0 and n - 1 others at `step` (in units of 2, rounded to the type), whose values are 1 and a little."""
    c = Cache([n], dtype, seed=5)
    rows = rows_at(c.table, 0, 0, n)
    x = 1 + 0.25 * torch.randn((n, 576), generator=gen(3), device=DEV)
    x[:, 512:] = 0.0
    x[:, 512] = step * math.log(2.0)
    x[at, :512], x[at, 512] = sink_value, 0.0
    c.pool.view(-1, 576)[rows] = x.to(T16[dtype])
    q = torch.zeros((1, heads, 576), dtype=T16[dtype], device=DEV)
    q[..., 512] = 1.0
    return c, q, [torch.ones((heads, n), dtype=torch.bool, device=DEV)]


def share_depth(n, sms):
    """Additions that a key of a sequence over all SMs goes through: its piece's keys and a page more, and the pieces."""
    return n // sms + 128 + sms


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("step", [-25.0, -24.6, -20.3])
@pytest.mark.parametrize("at", [0, 317])
def test_many_keys_far_below_one(dtype, step, at):
    n, sms = 131073, ops.num_sms()
    c, q, seen = sink_case(n, step, 1.0, dtype, at=at)
    out, lse = decode(c, q, scale=1.0)
    check(c, q, 1.0, out, lse, seen, 1, share_depth(n, sms))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("step", [-25.0, -24.6])
def test_many_keys_of_larger_values_far_below_one_in_one_piece(dtype, step):
    """A sixth of the output comes from keys at 2^-25 of the one beside them, all in one CTA's piece."""
    n = 131073
    c, q, seen = sink_case(n, step, 1.0, dtype)
    rows = rows_at(c.table, 0, 0, n)
    c.pool.view(-1, 576)[rows[torch.arange(n, device=DEV) != 317], :512] *= 50.0
    out, lse = decode(c, q, scale=1.0, sms=1)
    check(c, q, 1.0, out, lse, seen, 1, n // 8)  # (two roundings for each 16 keys)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("share", [0.01, 0.003])
@pytest.mark.parametrize("sms", [1, 20, None])
def test_a_long_light_tail_beside_a_key_of_no_value(dtype, share, sms):
    """The tail's values are all that is left in the output."""
    n = 65537 if sms is None else 20000
    c, q, seen = sink_case(n, math.log2(share / (n - 1)), 0.0, dtype)
    out, lse = decode(c, q, scale=1.0, sms=sms)
    check(c, q, 1.0, out, lse, seen, 1, share_depth(n, sms or ops.num_sms()))


# ----------------------------------------------------------------- long sequences, page by page

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [8, 20, 128])
def test_every_page_of_a_long_sequence_shows(dtype, heads):
    """Page p is all that column p % 512 holds but for pages a multiple of 512 away, whose values are others: a page lost,
    doubled or taken for another one is off by at least a sixth of its column."""
    n, sms = 70000, ops.num_sms()
    c = Cache([n], dtype, seed=6)
    rows = rows_at(c.table, 0, 0, n)
    x = torch.zeros((n, 576), device=DEV)
    page = torch.arange(n, device=DEV) // 64
    x[torch.arange(n, device=DEV), page % 512] = 2.0 + page // 512
    x[:, 512:] = torch.randn((n, 64), generator=gen(4), device=DEV)
    c.pool.view(-1, 576)[rows] = x.to(T16[dtype])
    q = normal((1, heads, 576), 2, dtype)
    q[..., :512] = 0.0
    blocks = -(-heads // (16 if heads <= 16 else 32 if heads <= 32 else 64))
    seen = [torch.ones((heads, n), dtype=torch.bool, device=DEV)]
    check(c, q, SCALE, *decode(c, q), seen, 64, share_depth(n, sms // blocks))
