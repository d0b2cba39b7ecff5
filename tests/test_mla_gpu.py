"""The latent cache on the GPU: both head products, append, gather and decode
against fp64, what lies outside a call untouched, and the calls run together
against attention over expanded keys and values."""
import math

import numpy as np
import pytest
import torch

from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops
from paged_kv_attention_fwd_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda"
T16 = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # a rounding, relative
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25}      # and below the type's normal range
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, seed, dtype="bf16"):
    return torch.randn(shape, generator=gen(seed), device=DEV).to(T16[dtype])


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEV)


def ok(workspace):
    assert B.pa_check_status(workspace) == B.PA_OK, B.pa_last_error()


def turned(x, at, table, interleaved):
    """fp64: every pair of x [T, ..., 64] turned by its angle of row at[t]."""
    x, w = x.double(), table.double()[at.long()].reshape(at.shape[0], *[1] * (x.dim() - 2), 64)
    c, s = w[..., :32], w[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    a, b = a * c - b * s, b * c + a * s
    return torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)


def near(got, want, tol):
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), f"off by {(off / tol).max():.3g} of the tolerance"


# ----------------------------------------------------------------- the head products

def product_tol(want, reach, terms, dtype):
    """One rounding, and `terms` fp32 sums (2^-23 each, truncation included) of products whose magnitudes sum to reach."""
    return HALF[dtype] * want.abs() + terms * 2.0 ** -23 * reach + TINY[dtype]


@pytest.mark.parametrize("t,h", [(1, 1), (2, 3), (17, 8), (127, 2), (128, 1), (129, 5), (300, 3), (700, 1)])
@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("f16", True)])
def test_query_against_fp64(t, h, dtype, inter):
    packed = normal((t, h * 192 + 40), 1, dtype)
    q = packed[:, 8:8 + h * 192].unflatten(-1, (h, 192))
    w = (normal((h, 256, 512), 2, dtype) * 0.05)[:, :128]
    at = torch.randint(0, 500, (t,), generator=gen(3), device=DEV, dtype=torch.int32)
    table = ops.rope_table(500, 64)
    room = torch.full((t + 1, h * 576 + 16), 7.0, dtype=T16[dtype], device=DEV)
    out = room[:t, :h * 576].unflatten(-1, (h, 576))
    _, ws = ops.mla_query(q, w, at, table, inter, q_out=out)
    ok(ws)
    want = torch.einsum("thi,hik->thk", q[..., :128].double(), w.double())
    reach = torch.einsum("thi,hik->thk", q[..., :128].double().abs(), w.double().abs())
    near(out[..., :512], want, product_tol(want, reach, 128, dtype))
    want = turned(q[..., 128:], at, table, inter)
    near(out[..., 512:], want, HALF[dtype] * want.abs() + 2.0 ** -22 * q[..., 128:].double().abs().amax() + TINY[dtype])
    assert (room[t] == 7).all() and (room[:, h * 576:] == 7).all()


@pytest.mark.parametrize("t,h,dtype,inter", [(2100, 64, "f16", True), (40, 304, "bf16", False), (200, 300, "bf16", True)])
def test_query_many_tiles_a_head_and_many_heads(t, h, dtype, inter):
    """Enough heads and tokens that an SM goes through several tiles of a head, or through several heads."""
    test_query_against_fp64(t, h, dtype, inter)


def test_query_padding_bad_positions_and_no_rotation():
    t, h = 140, 2
    q, w, table = normal((t, h, 192), 1), normal((h, 128, 512), 2) * 0.05, ops.rope_table(50, 64)
    at = torch.arange(t, device=DEV, dtype=torch.int32) % 50
    want, ws = ops.mla_query(q, w, at, table)
    ok(ws)
    q2 = q.clone()
    at2 = at.clone()
    at2[[0, 130]], at2[7] = -3, 50
    q2[[0, 7, 130]] = float("nan")
    out = torch.full_like(want, 5.0)
    _, ws = ops.mla_query(q2, w, at2, table, q_out=out)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    rest = torch.ones(t, dtype=torch.bool, device=DEV)
    rest[[0, 7, 130]] = False
    assert (out[~rest] == 5).all() and torch.equal(out[rest], want[rest])
    out, ws = ops.mla_query(q, w)
    ok(ws)
    assert torch.equal(out[..., 512:], q[..., 128:]) and torch.equal(out[..., :512], want[..., :512])


@pytest.mark.parametrize("t,h", [(1, 1), (3, 2), (64, 8), (128, 3), (129, 2), (513, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_output_against_fp64(t, h, dtype):
    o = normal((t, h * 512 + 8), 1, dtype)[:, :h * 512].unflatten(-1, (h, 512))
    w = (normal((h, 256, 512), 2, dtype) * 0.05)[:, 128:]
    room = torch.full((t + 1, h * 128 + 8), 7.0, dtype=T16[dtype], device=DEV)
    out = room[:t, :h * 128].unflatten(-1, (h, 128))
    _, ws = ops.mla_output(o, w, out)
    ok(ws)
    want = torch.einsum("thk,hik->thi", o.double(), w.double())
    reach = torch.einsum("thk,hik->thi", o.double().abs(), w.double().abs())
    near(out, want, product_tol(want, reach, 512, dtype))
    assert (room[t] == 7).all() and (room[:, h * 128:] == 7).all()


@pytest.mark.parametrize("t,h,dtype", [(1500, 32, "f16"), (40, 304, "bf16"), (1000, 200, "bf16"), (20000, 1, "bf16"), (300, 100, "f16")])
def test_output_many_tiles_a_head_and_many_heads(t, h, dtype):
    """Shares of an SM that hold several tiles, parts of tiles, and several heads' weights."""
    test_output_against_fp64(t, h, dtype)


def test_products_keep_nan_to_its_token_and_head():
    q, o, w = normal((200, 3, 192), 1), normal((200, 3, 512), 2), normal((3, 128, 512), 3)
    a, b = ops.mla_query(q, w)[0], ops.mla_output(o, w)[0]
    q[150, 1], o[20, 2], w[0] = float("nan"), float("inf"), float("nan")
    a2, b2 = ops.mla_query(q, w)[0], ops.mla_output(o, w)[0]
    assert a2[:, 0, :512].isnan().all() and b2[:, 0].isnan().all()
    keep = torch.ones((200, 3), dtype=torch.bool, device=DEV)
    keep[:, 0] = False
    ka, kb = keep.clone(), keep.clone()
    ka[150, 1] = kb[20, 2] = False
    assert torch.equal(a2[ka], a[ka]) and torch.equal(b2[kb], b[kb])
    assert not a2[150, 1].isfinite().any() and not b2[20, 2].isfinite().any()


# ----------------------------------------------------------------- pages

def pages_of(lens, seed=0, extra=3, width=None):
    """A block table of pages in random order and the number of pages; unused slots hold what no call may read."""
    need = [-(-n // 64) for n in lens]
    total = sum(need) + extra
    order = np.random.default_rng(seed).permutation(total).astype(np.int32)
    table = np.full((len(lens), width or max(need + [1])), 2 ** 31 - 1, np.int32)
    first = 0
    for b, n in enumerate(need):
        table[b, :n] = order[first:first + n]
        first += n
    return torch.from_numpy(table).to(DEV), total


def rows_at(table, b, first, count):
    """Pool rows (page * 64 + row) of positions first .. first + count - 1 of sequence b."""
    p = torch.arange(first, first + count, device=DEV)
    return table[b, p // 64].long() * 64 + p % 64


@pytest.mark.parametrize("prior,new", [([0], [1]), ([63, 64, 65], [1, 1, 1]), ([5, 0, 130], [70, 0, 3]),
                                       (list(range(40)), [1 + b % 3 for b in range(40)]), ([7] * 200, [2] * 200)])
@pytest.mark.parametrize("dtype,inter", [("bf16", True), ("f16", False)])
def test_append_against_fp64(prior, new, dtype, inter):
    table, total = pages_of([p + n for p, n in zip(prior, new)])
    count, pad = sum(new), 5
    kv = normal((count + pad, 640), 1, dtype)[:, 64:]
    kv[count:] = float("nan")  # padding behind the last sequence
    weight = 1 + 0.2 * normal((512,), 2, dtype)
    angles = ops.rope_table(300, 64)
    pool = normal((total, 64, 576), 3, dtype)
    before = pool.clone()
    cu, start = ints(np.cumsum([0] + new)), ints(prior)
    sh = ops.mla_cache_shapes(len(new), table.shape[1], total, count + pad, dtype, kv, 300, inter, eps=1e-5)
    ok(ops.mla_append_kv(sh, kv, cu, start, table, pool, weight, None, angles))
    at = torch.cat([rows_at(table, b, p, n) for b, (p, n) in enumerate(zip(prior, new))])
    pos = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(prior, new)])
    x = kv[:count, :512].double()
    want = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * weight.double()
    got = pool.view(-1, 576)
    # 512 squares summed in fp32 (half of their relative error comes through the root), a root and two products
    near(got[at, :512], want, (HALF[dtype] + 2.0 ** -15) * want.abs() + TINY[dtype])
    want = turned(kv[:count, 512:], pos, angles, inter)
    near(got[at, 512:], want, HALF[dtype] * want.abs() + 2.0 ** -22 * 8 + TINY[dtype])
    rest = torch.ones(total * 64, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert torch.equal(got[rest], before.view(-1, 576)[rest])


def test_append_copies_where_nothing_is_asked_for():
    table, total = pages_of([70, 70])
    kv, pool = normal((6, 576), 1), ops.mla_pool(total)
    sh = ops.mla_cache_shapes(2, table.shape[1], total, 6, kv=kv, norm=False)
    ok(ops.mla_append_kv(sh, kv, ints([0, 2, 6]), ints([0, 62]), table, pool))
    got = pool.view(-1, 576)
    assert torch.equal(got[rows_at(table, 0, 0, 2)], kv[:2]) and torch.equal(got[rows_at(table, 1, 62, 4)], kv[2:])
    ok(ops.mla_append_kv(ops.mla_cache_shapes(2, table.shape[1], total, 6, kv=kv, eps=0.0), kv, ints([0, 2, 6]), ints([0, 62]),
                         table, pool))  # a norm without weights
    x = kv.double()
    want = x[:, :512] / x[:, :512].square().mean(-1, keepdim=True).sqrt()
    near(got[rows_at(table, 1, 62, 4), :512], want[2:], (HALF["bf16"] + 2.0 ** -15) * want[2:].abs())


def test_append_positions_padding_and_what_is_out_of_range():
    table, total = pages_of([64, 64, 64], width=2)
    kv = normal((6, 576), 1)
    angles = ops.rope_table(20, 64)
    pool = torch.full((total, 64, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    # token 1 is padding by its position, 2 past the angles, 4 past the table's row, 5 on a page that is none
    at = ints([4, -1, 20, 0, 1, 2])
    sh = ops.mla_cache_shapes(3, 2, total, 6, kv=kv, max_position=20, norm=False)
    table[2, 1] = total
    ws = ops.mla_append_kv(sh, kv, ints([0, 3, 5, 6]), ints([0, 127, 64]), table, pool, None, at, angles)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    got = pool.view(-1, 576)
    touched = (got != 3).any(-1).nonzero().flatten()
    assert touched.tolist() == rows_at(table, 0, 0, 1).tolist()  # (sequence 1's page 1 is 2^31 - 1: none)
    assert torch.equal(got[touched[0], :512], kv[0, :512])
    want = turned(kv[:1, 512:], at[:1], angles, False)
    near(got[touched, 512:], want, HALF["bf16"] * want.abs() + 2.0 ** -19)


@pytest.mark.parametrize("first,count", [([0], [1]), ([3, 60, 0], [61, 70, 0]), (list(range(50)), [1 + b % 9 for b in range(50)])])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gather_bit_for_bit(first, count, dtype):
    table, total = pages_of([f + c for f, c in zip(first, count)])
    pool = torch.randint(-2 ** 15, 2 ** 15, (total, 64, 576), generator=gen(1), device=DEV, dtype=torch.int16).view(T16[dtype])
    n, pad = sum(count), 3
    sh = ops.mla_cache_shapes(len(first), table.shape[1], total, n + pad, dtype)
    latent = torch.full((n + pad, 512), 9.0, dtype=T16[dtype], device=DEV)
    rope = torch.full((n + pad, 1, 64), 9.0, dtype=T16[dtype], device=DEV)
    _, _, ws = ops.mla_gather_kv(sh, pool, ints(np.cumsum([0] + count)), ints(first), table, latent, rope)
    ok(ws)
    want = pool.view(torch.int16).view(-1, 576)[torch.cat([rows_at(table, b, f, c) for b, (f, c) in enumerate(zip(first, count))])]
    assert torch.equal(latent.view(torch.int16)[:n], want[:, :512]) and torch.equal(rope.view(torch.int16)[:n, 0], want[:, 512:])
    assert (latent[n:] == 9).all() and (rope[n:] == 9).all()


def test_gather_of_what_is_out_of_range_leaves_its_rows():
    table, total = pages_of([64, 64], width=1)
    table[1, 0] = -5
    pool = normal((total, 64, 576), 1)
    sh = ops.mla_cache_shapes(2, 1, total, 6)
    latent, rope = (torch.full(s, 9.0, dtype=torch.bfloat16, device=DEV) for s in ((6, 512), (6, 1, 64)))
    _, _, ws = ops.mla_gather_kv(sh, pool, ints([0, 3, 6]), ints([62, 0]), table, latent, rope)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    want = pool.view(-1, 576)[rows_at(table, 0, 62, 2)]
    assert torch.equal(latent[:2], want[:, :512]) and (latent[2:] == 9).all() and (rope[2:] == 9).all()


# ----------------------------------------------------------------- decode

class Cache:
    def __init__(self, lens, dtype="bf16", seed=0, gain=1.0, width=None):
        self.lens, self.dtype = list(lens), dtype
        self.table, self.total = pages_of(lens, seed, width=width)
        self.pool = (torch.randn((self.total, 64, 576), generator=gen(seed + 10), device=DEV) * gain).to(T16[dtype])
        live = torch.zeros(self.total * 64, dtype=torch.bool, device=DEV)
        for b, n in enumerate(self.lens):
            live[rows_at(self.table, b, 0, n)] = True
        self.pool.view(-1, 576)[~live] = float("nan")  # rows that belong to nobody

    def rows(self, b):
        return self.pool.view(-1, 576)[rows_at(self.table, b, 0, self.lens[b])].double()

    def shapes(self, heads, q_len=1, sms=None):
        return ops.mla_decode_shapes(len(self.lens), heads, self.table.shape[1], self.total, q_len, self.dtype, sms=sms)


def check_decode(c, q, scale, out, lse, q_len=1, skip=()):
    h = q.shape[1]
    out, lse = out.double(), lse.double()
    for b, n in enumerate(c.lens):
        if b in skip:
            continue
        k = c.rows(b)
        for i in range(q_len):
            t, sees = b * q_len + i, max(0, n - (q_len - 1 - i))
            if sees == 0:
                assert (out[t] == 0).all() and (lse[t] == -math.inf).all()
                continue
            s = q[t].double() @ k[:sees].T * scale
            reach = (q[t].double().abs() @ k[:sees].abs().T * abs(scale)).amax(-1)
            want = torch.logsumexp(s, -1)
            p = torch.exp(s - want[:, None])
            o, spread = p @ k[:sees, :512], p @ k[:sees, :512].abs()
            # a score: 576 fp32 products and the steps up to the exponent (2^-23 of its reach each), the exponential 2^-21
            logit = ((576 + 4) * 2.0 ** -23 * reach + 2.0 ** -21)[:, None]
            # weights: half a step each, below fp16's normal range 2^-25 of the reference's, whose own weight is 1
            below = sees * 2.0 ** -25 * k[:sees, :512].abs().amax() if c.dtype == "f16" else 0.0
            tol = HALF[c.dtype] * o.abs() + (HALF[c.dtype] + 2 * logit + sees * 2.0 ** -24) * spread + below + TINY[c.dtype]
            assert torch.isfinite(out[t]).all()
            assert ((out[t] - o).abs() <= tol).all(), (b, i, ((out[t] - o).abs() / tol).max().item())
            ltol = logit[:, 0] + sees * 2.0 ** -24 + 2.0 ** -22 * (want.abs() + 1)
            assert ((lse[t] - want).abs() <= ltol).all(), (b, i, ((lse[t] - want).abs() / ltol).max().item())


def decode(c, q, q_len=1, scale=SCALE, sms=None, **more):
    out, lse, ws = ops.mla_decode(c.shapes(q.shape[1], q_len, sms), q, c.pool, c.table, ints(c.lens), scale, **more)
    ok(ws)
    return out, lse


@pytest.mark.parametrize("heads", [1, 5, 16, 17, 32, 33, 64, 65, 128, 130])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_heads(heads, dtype):
    c = Cache([300, 0, 64, 1, 1000], dtype)
    q = normal((5, heads, 576), 1, dtype)
    check_decode(c, q, SCALE, *decode(c, q))


@pytest.mark.parametrize("q_len,heads", [(2, 16), (3, 5), (4, 32), (2, 128), (7, 9)])
def test_decode_of_several_tokens(q_len, heads):
    c = Cache([300, 0, 1, 2, 64, 65, 63, 3, 700], "bf16", seed=q_len)
    q = normal((9 * q_len, heads, 576), 1)
    check_decode(c, q, SCALE, *decode(c, q, q_len), q_len)


@pytest.mark.parametrize("heads,q_len", [(16, 1), (40, 1), (8, 2)])
def test_decode_every_short_length(heads, q_len):
    c = Cache(range(1, 200), "bf16", seed=3)
    q = normal((199 * q_len, heads, 576), 1)
    check_decode(c, q, SCALE, *decode(c, q, q_len), q_len)


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 40, None])
@pytest.mark.parametrize("lens,heads", [([1500], 128), ([130, 4000, 20, 999], 64), ([5] * 90 + [3000] + [0] * 40, 16)])
def test_decode_dealt_to_any_number_of_sms(sms, lens, heads):
    c = Cache(lens, "bf16", seed=4)
    q = normal((len(lens), heads, 576), 1)
    check_decode(c, q, SCALE, *decode(c, q, sms=sms))


def test_decode_one_long_sequence_and_many_short_ones():
    c = Cache([70000], "f16", seed=5)
    q = normal((1, 20, 576), 1, "f16")
    check_decode(c, q, SCALE, *decode(c, q))
    c = Cache([i % 4 for i in range(3000)], "bf16", seed=6)
    q = normal((3000, 4, 576), 1)
    check_decode(c, q, SCALE, *decode(c, q))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale,gain", [(SCALE, 6.0), (-SCALE, 1.0), (0.0, 1.0), (1.0, 1.0)])
def test_decode_scales(dtype, scale, gain):
    c = Cache([900, 100], dtype, gain=gain)
    q = normal((2, 24, 576), 1, dtype)
    check_decode(c, q, scale, *decode(c, q, scale=scale))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [16, 32, 64])
def test_decode_growing_maximum(dtype, heads):
    """Scores that rise from page to page by up to 2^40, for some columns only."""
    c = Cache([1300, 700], dtype)
    for b, n in enumerate(c.lens):
        at = rows_at(c.table, b, 0, n)
        step = (torch.arange(n, device=DEV) // 50).to(T16[dtype])
        c.pool.view(-1, 576)[at, 500] = step
    q = normal((2, heads, 576), 1, dtype)
    q[:, ::3, 500] = 14.0
    q[:, 1::3, 500] = -14.0
    check_decode(c, q, SCALE, *decode(c, q))


def test_decode_nan_reaches_its_sequence_and_head_only():
    c = Cache([200, 300, 70])
    q = normal((3, 20, 576), 1)
    out, lse = decode(c, q)
    c.pool.view(-1, 576)[rows_at(c.table, 1, 130, 1), 7] = float("nan")
    q[2, 5] = float("inf")
    out2, lse2 = decode(c, q)
    assert out2[1].isnan().all() and not out2[2, 5].isfinite().any()
    keep = torch.ones((3, 20), dtype=torch.bool, device=DEV)
    keep[1], keep[2, 5] = False, False
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[keep], lse[keep])


def test_decode_of_a_dominant_key_and_of_minus_infinity():
    c = Cache([500], "f16")
    q = torch.zeros((1, 16, 576), dtype=torch.float16, device=DEV)
    q[0, :, 0] = 60.0
    at = rows_at(c.table, 0, 0, 500)
    c.pool.view(-1, 576)[at, 0] = -60.0
    c.pool.view(-1, 576)[at[317], 0] = 60.0
    check_decode(c, q, 1.0, *decode(c, q, scale=1.0))
    # scores of -inf weigh nothing, wherever they stand (their values are what the weights multiply: finite here)
    c = Cache([200])
    at = rows_at(c.table, 0, 0, 200)
    q = normal((1, 8, 576), 1)
    q[..., 575] = 1.0
    hidden = torch.arange(0, 200, 3, device=DEV)
    c.pool.view(-1, 576)[at[hidden], 575] = -float("inf")
    out, lse = decode(c, q)
    seen = torch.ones(200, dtype=torch.bool, device=DEV)
    seen[hidden] = False
    k = c.rows(0)[seen]
    s = q[0].double() @ k.T * SCALE
    near(lse[0], torch.logsumexp(s, -1), torch.full((8,), 1e-4, device=DEV, dtype=torch.float64))
    o, spread = torch.softmax(s, -1) @ k[:, :512], torch.softmax(s, -1) @ k[:, :512].abs()
    near(out[0], o, HALF["bf16"] * (o.abs() + spread) + 1e-3 * spread)


def test_decode_repeats_bit_for_bit_whatever_the_page_order():
    c = Cache([3000, 17, 640, 1], seed=7)
    q = normal((4, 128, 576), 1)
    out, lse = decode(c, q)
    for _ in range(3):
        o, l = decode(c, q)
        assert torch.equal(o, out) and torch.equal(l, lse)
    perm = torch.randperm(c.total, generator=gen(2), device=DEV)
    pool = torch.empty_like(c.pool)
    pool[perm] = c.pool
    live = c.table < c.total
    c.table[live] = perm[c.table[live].long()].to(torch.int32)
    c.pool = pool
    o, l = decode(c, q)
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_decode_reports_bad_pages_and_lengths():
    c = Cache([200, 300, 100], width=5)
    q = normal((3, 32, 576), 1)
    table = c.table.clone()
    table[1, 2] = c.total
    out, lse, ws = ops.mla_decode(c.shapes(32), q, c.pool, table, ints(c.lens), SCALE)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    check_decode(c, q, SCALE, out, lse, skip=(1,))
    for bad in (-1, 5 * 64 + 1):
        lens = ints([200, bad, 100])
        table[1] = c.table[0, 0]
        out, lse, ws = ops.mla_decode(c.shapes(32), q, c.pool, table, lens, SCALE)
        assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
        check_decode(c, q, SCALE, out, lse, skip=(1,))
        if bad < 0:
            assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_decode_writes_its_rows_only_and_may_leave_out_lse():
    c = Cache([130, 700])
    q = normal((2, 48, 576), 1)
    want, _ = decode(c, q)
    sh = c.shapes(48)
    room = torch.full((2 * 48 * 512 + 1024,), 7.0, dtype=torch.bfloat16, device=DEV)
    size = B.pa_mla_decode_workspace_size(sh)
    ws = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)  # stale contents behind the status word
    ws[:B.PA_STATUS_BYTES] = 0
    B.pa_mla_decode(sh, q, c.pool, c.table, ints(c.lens), SCALE, room[512:], None, ws, size)
    ok(ws)
    assert torch.equal(room[512:-512].view(2, 48, 512), want)
    assert (room[:512] == 7).all() and (room[-512:] == 7).all() and (ws[size:] == 0xA5).all()


def test_captured_decode_follows_new_lengths_tables_and_queries():
    caches = [Cache(l, seed=i, width=40) for i, l in enumerate(([2500, 10, 0, 640], [1, 2000, 63, 64], [0, 0, 0, 5]))]
    total = max(c.total for c in caches)
    sh = ops.mla_decode_shapes(4, 128, 40, total)
    q, lens, table = normal((4, 128, 576), 1), ints(caches[0].lens), caches[0].table.clone()
    pool = torch.zeros((total, 64, 576), dtype=torch.bfloat16, device=DEV)
    out, lse, ws = ops.mla_decode(sh, q, pool, table, lens, SCALE)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.mla_decode(sh, q, pool, table, lens, SCALE, out, lse, ws)
    for i, c in enumerate(caches):
        pool[:c.total].copy_(c.pool)
        table.copy_(c.table)
        lens.copy_(ints(c.lens))
        q.copy_(normal((4, 128, 576), 20 + i))
        graph.replay()
        ok(ws)
        check_decode(c, q, SCALE, out, lse)


def test_pages_past_two_to_the_31_elements():
    """A 5 GB pool: rows appended behind 2^31 elements (2^32 bytes), attended over and read back."""
    pages, n, heads = 70000, 200, 24
    pool = torch.full((pages, 64, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = ints([[pages - 1, 59000, 58500, pages - 7]])
    kv = normal((n, 576), 1)
    sh = ops.mla_cache_shapes(1, 4, pages, n, norm=False)
    ok(ops.mla_append_kv(sh, kv, ints([0, n]), ints([0]), table, pool))
    assert torch.equal(pool.view(-1, 576)[rows_at(table, 0, 0, n)], kv)
    latent, rope, ws = ops.mla_gather_kv(sh, pool, ints([0, n]), ints([0]), table)
    ok(ws)
    assert torch.equal(latent, kv[:, :512]) and torch.equal(rope[:, 0], kv[:, 512:])
    q = normal((1, heads, 576), 2)
    out, lse, ws = ops.mla_decode(ops.mla_decode_shapes(1, heads, 4, pages), q, pool, table, ints([n]), SCALE)
    ok(ws)
    near_pages = Cache([n], "bf16")  # the same rows in pages at the front
    near_pages.pool.view(-1, 576)[rows_at(near_pages.table, 0, 0, n)] = kv
    want = decode(near_pages, q)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    check_decode(near_pages, q, SCALE, out, lse)


def test_calls_of_other_shapes_share_a_dirty_workspace():
    """One after the other: few long sequences, many short ones, none with a key, one block and several."""
    cases = [([9000], 128), ([70, 0, 5000] + [3] * 60, 16), ([0, 0, 0], 40), ([4000, 1], 20), ([65] * 20, 128), ([9000], 128)]
    caches = [Cache(lens, "bf16", seed=20 + i, width=150) for i, (lens, _) in enumerate(cases)]
    need = max(B.pa_mla_decode_workspace_size(c.shapes(h)) for c, (_, h) in zip(caches, cases))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ws[:B.PA_STATUS_BYTES] = 0
    for c, (lens, h) in zip(caches, cases):
        q = normal((len(lens), h, 576), 1)
        check_decode(c, q, SCALE, *decode(c, q, workspace=ws))


def test_two_streams_with_their_own_workspaces():
    caches = [Cache([1500, 900, 30], seed=i) for i in (1, 2)]
    qs = [normal((3, 64, 576), i) for i in (3, 4)]
    want = [decode(c, q) for c, q in zip(caches, qs)]
    streams = [torch.cuda.Stream() for _ in caches]
    lens = [ints(c.lens) for c in caches]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append([ops.mla_decode(c.shapes(64), q, c.pool, c.table, n, SCALE, stream=s)
                    for c, q, n, s in zip(caches, qs, lens, streams)])
    torch.cuda.synchronize()
    for pair in got:
        for (out, lse, ws), (o, l) in zip(pair, want):
            ok(ws)
            assert torch.equal(out, o) and torch.equal(lse, l)


# ----------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("f16", True)])
def test_steps_against_attention_over_expanded_keys(dtype, inter):
    """A prompt appended and read back for the expanded prefill, then single tokens appended and attended over in the
    absorbed form: both against fp64 over expanded keys and values."""
    h, prompts, steps, dt = 4, [70, 1, 200], 3, T16[dtype]
    table, total = pages_of([p + steps for p in prompts])
    pool = ops.mla_pool(total, dtype)
    packed = normal((h, 256, 512), 1, dtype) * 512 ** -0.5
    w_uk, w_uv = packed[:, :128], packed[:, 128:]
    weight = (1 + 0.1 * normal((512,), 2, dtype)).to(dt)
    angles = ops.rope_table(512, 64)
    cached = [torch.empty((0, 576), dtype=torch.float64, device=DEV) for _ in prompts]
    start = [0] * len(prompts)

    def append(counts, seed):
        kv = normal((sum(counts), 576), seed, dtype)
        sh = ops.mla_cache_shapes(len(prompts), table.shape[1], total, sum(counts), dtype, kv, 512, inter)
        ok(ops.mla_append_kv(sh, kv, ints(np.cumsum([0] + counts)), ints(start), table, pool, weight, None, angles))
        for b, n in enumerate(counts):
            start[b] += n
            cached[b] = pool.view(-1, 576)[rows_at(table, b, 0, start[b])].double()

    def expanded(b):
        c = cached[b][:, :512]
        k = torch.einsum("nk,hik->hni", c, w_uk.double())
        return (torch.cat((k, cached[b][:, None, 512:].expand(-1, h, -1).transpose(0, 1)), -1),
                torch.einsum("nk,hik->hni", c, w_uv.double()))

    append(prompts, 5)
    # the expanded prefill over rows read back
    cu = ints(np.cumsum([0] + prompts))
    sh = ops.mla_cache_shapes(len(prompts), table.shape[1], total, sum(prompts), dtype)
    latent, rope, ws = ops.mla_gather_kv(sh, pool, cu, ints([0] * 3), table)
    ok(ws)
    k = (latent @ w_uk.flatten(0, 1).T).unflatten(-1, (h, 128))
    v = (latent @ w_uv.flatten(0, 1).T).unflatten(-1, (h, 128))
    q = normal((sum(prompts), h, 192), 6, dtype)
    pos = torch.cat([torch.arange(n, device=DEV) for n in prompts]).to(torch.int32)
    q_turned = torch.cat((q[..., :128], turned(q[..., 128:], pos, angles, inter).to(dt)), -1)
    psh = ops.prefill_shapes(3, h, h, 192, 128, 64, max(prompts), sum(prompts), sum(prompts), dtype=dtype)
    out, _, ws = ops.prefill(psh, q_turned, k.contiguous(), v.contiguous(), cu, cu, SCALE, True, k_rope=rope)
    ok(ws)
    t = 0
    for b, n in enumerate(prompts):
        kk, vv = expanded(b)
        s = torch.einsum("thi,hni->htn", q_turned[t:t + n].double(), kk) * SCALE
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -math.inf)
        want = torch.einsum("htn,hni->thi", torch.softmax(s, -1), vv)
        # keys, values, weights and the result each rounded once; a score moves by its rounded key's share
        assert (out[t:t + n].double() - want).abs().max() <= 16 * HALF[dtype]
        t += n
    # single tokens, absorbed
    for step in range(steps):
        append([1, 1, 1], 10 + step)
        q = normal((3, h, 192), 20 + step, dtype)
        q_lat, ws = ops.mla_query(q, w_uk, ints([n - 1 for n in start]), angles, inter)
        ok(ws)
        dsh = ops.mla_decode_shapes(3, h, table.shape[1], total, dtype=dtype)
        o, _, ws = ops.mla_decode(dsh, q_lat, pool, table, ints(start), SCALE)
        ok(ws)
        out, ws = ops.mla_output(o, w_uv)
        ok(ws)
        for b, n in enumerate(start):
            kk, vv = expanded(b)
            qq = torch.cat((q[b, :, :128].double(), turned(q[b:b + 1, :, 128:], ints([n - 1]), angles, inter)[0]), -1)
            s = torch.einsum("hi,hni->hn", qq, kk) * SCALE
            want = torch.einsum("hn,hni->hi", torch.softmax(s, -1), vv)
            assert (out[b].double() - want).abs().max() <= 16 * HALF[dtype]


def test_whole_step_captured_and_on_a_given_stream():
    """query, append, decode and output in one graph, replayed with new tokens, against the calls one by one."""
    h, lens = 16, [100, 64, 1]
    table, total = pages_of([n + 4 for n in lens])
    pools = [normal((total, 64, 576), 1) for _ in range(2)]
    w = normal((h, 256, 512), 2) * 0.05
    angles = ops.rope_table(256, 64)
    q, kv = normal((3, h, 192), 3), normal((3, 576), 4)
    start, after, at = ints(lens), ints([n + 1 for n in lens]), ints(lens)
    cu = ints([0, 1, 2, 3])
    csh = ops.mla_cache_shapes(3, table.shape[1], total, 3, kv=kv, max_position=256)
    dsh = ops.mla_decode_shapes(3, h, table.shape[1], total)

    def step(pool, **stream):
        q_lat, ws1 = ops.mla_query(q, w[:, :128], at, angles, **stream)
        ws2 = ops.mla_append_kv(csh, kv, cu, start, table, pool, None, None, angles, **stream)
        o, lse, ws3 = ops.mla_decode(dsh, q_lat, pool, table, after, SCALE, **stream)
        out, ws4 = ops.mla_output(o, w[:, 128:], **stream)
        return out, lse, (ws1, ws2, ws3, ws4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(pools[0], stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(pools[0])
    for i in range(3):
        q.copy_(normal((3, h, 192), 30 + i))
        kv.copy_(normal((3, 576), 40 + i))
        start.copy_(ints([n + i for n in lens]))
        at.copy_(start)
        after.copy_(start + 1)
        graph.replay()
        want = step(pools[1])
        torch.cuda.synchronize()
        for ws in got[2] + want[2]:
            ok(ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
