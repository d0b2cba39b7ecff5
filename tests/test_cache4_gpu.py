"""4-bit pages on the GPU: pa_append_kv and pa_gather_kv bit for bit against
the plain forms, and pa_decode over 4-bit pages against fp64."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp4 as F
from oracle import scheduler as S
from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops
from paged_kv_attention_fwd_gb300 import workloads as W
from paged_kv_attention_fwd_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def heads(hk, seed=0):
    return (0.003 + 0.01 * np.random.default_rng(seed).random(hk)).astype(np.float32)


class Cache:
    """A 4-bit cache on the host (bytes and float64 values) and on the device."""

    def __init__(self, lens, hk, d, seed=0, room=0, extra=3, max_pages=None):
        lens = np.asarray(lens, np.int32)
        self.lens, self.hk, self.d = lens, hk, d
        self.table, self.pages = W.assign_pages(lens + room, seed, extra, max_pages)
        shape = (self.pages, hk, 64, d)
        n = int(np.prod(shape))
        self.ks, self.vs = heads(hk, seed), heads(hk, seed + 1)
        self.k = F.make_pool(W.normal_f32(seed, 60, n).reshape(shape), self.ks)
        self.v = F.make_pool(W.normal_f32(seed, 61, n).reshape(shape), self.vs)

    def poison(self):
        """NaN scales and saturated codes wherever no live key lies."""
        for pool in (self.k, self.v):
            live = np.zeros((self.pages, 64), bool)
            for b, n in enumerate(self.lens):
                for i in range((n + 63) // 64):
                    live[self.table[b, i], : min(64, n - 64 * i)] = True
            codes, scales = F.rows_of_slab(pool, self.d)
            at = np.nonzero(~live)
            codes[at[0], :, at[1]] = 0xFF
            scales[at[0], :, at[1]] = 0x7F
        for b, n in enumerate(self.lens):  # slots past the sequence are never read
            self.table[b, (n + 63) // 64:] = 2 ** 31 - 1

    def up(self):
        return dev(self.k), dev(self.v), dev(self.ks), dev(self.vs), dev(self.table), dev(self.lens)

    def values(self):
        return F.decode_pool(self.k, self.ks, self.d), F.decode_pool(self.v, self.vs, self.d)


def check(c, q, scale, out, lse):
    """Out within its bf16 rounding, P's fp16 rounding and the logits' fp32 sums."""
    kv, vv = c.values()
    if np.isnan(kv).any() or np.isnan(vv).any():  # poisoned slots: never part of a sum
        kv, vv = np.nan_to_num(kv), np.nan_to_num(vv)
    ro, rl, spread, reach, top = F.attend(q, kv, vv, c.table, c.lens, scale)
    # a logit is a sum of D fp32 products (2^-23 each, truncation included); q itself is exact but for elements
    # below 2^-14 of the head's largest
    logit = (c.d * 2.0 ** -23 * reach + 2.0 ** -20)[..., None]
    # P: fp16, half a step 2^-11 relative, 2^-25 absolute per key below its normal range
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * logit) * spread + c.lens[:, None, None] * 2.0 ** -25 * top + 1e-30
    out = out.float().cpu().numpy()
    assert np.isfinite(out).all()
    assert (np.abs(out - ro) <= tol).all(), float((np.abs(out - ro) / tol).max())
    lse = lse.cpu().numpy()
    some = c.lens > 0
    assert np.all(lse[~some] == -np.inf) and np.all(out[~some] == 0)
    assert (np.abs(lse[some] - rl[some]) <= logit[some, :, 0] + 2.0 ** -20 * (1 + np.abs(rl[some]))).all()


def decode(c, hq, scale=None, seed=0, gain=1.0, **plan):
    scale = c.d ** -0.5 if scale is None else scale
    q = W.f32_to_bf16_bits(gain * W.normal_f32(seed, 62, len(c.lens) * hq * c.d)).reshape(len(c.lens), hq, c.d)
    p = ops.plan_decode(c.lens, None, hq, c.hk, c.d, c.table.shape[1], c.pages, kv_dtype="fp4", **plan)
    k, v, ks, vs, table, lens = c.up()
    out, lse = ops.decode(p, ops.as_bf16(q, DEV), k, v, table, lens, scale, ks, vs)
    assert B.pa_check_status(p.workspace) == B.PA_OK, B.pa_last_error()
    return q, scale, out, lse, p


# ----------------------------------------------------------------- append and read-back

@pytest.mark.parametrize("d,hk", [(128, 4), (128, 1), (128, 5), (128, 9), (64, 8), (64, 3)])
def test_append_bit_exact(d, hk):
    prior, new = np.array([0, 63, 64, 130, 1000], np.int32), np.array([5, 1, 70, 200, 64], np.int32)
    c = Cache(prior, hk, d, seed=70, room=new)
    cu = W.cu_seqlens(new)
    kn, vn = (W.bf16_normal(70, s, (int(cu[-1]), hk, d)) for s in (90, 91))
    kn[3, 0, :16] = 0                                       # an all-zero block
    kn[4, 0, 5] = 0x7F80                                    # +inf saturates
    kn[5, 0, 20] = 0x7FC0                                   # a NaN poisons its block
    vn[6, 0] = W.f32_to_bf16_bits(np.full(d, 1e30, np.float32))   # a saturated scale
    vn[7, 0] = W.f32_to_bf16_bits(np.full(d, 1e-38, np.float32))  # a scale that rounds to zero
    k, v, ks, vs, table, _ = c.up()
    sh = ops.append_shapes(len(prior), hk, d, c.table.shape[1], c.pages, int(cu[-1]), "fp4")
    ws = ops.append_kv(sh, ops.as_bf16(kn, DEV), ops.as_bf16(vn, DEV), dev(cu), dev(prior), table, k, v, ks, vs)
    assert B.pa_check_status(ws) == B.PA_OK
    assert np.array_equal(k.cpu().numpy(), F.append(kn, cu, prior, c.table, c.k, c.ks, d))
    assert np.array_equal(v.cpu().numpy(), F.append(vn, cu, prior, c.table, c.v, c.vs, d))


def test_codes_of_every_bf16_magnitude():
    """Every finite bf16 value next to a block maximum, for head scales whose
    products with a block scale are no round numbers: the codes are those of
    the fp32 quotient."""
    d, hk, t = 128, 8, 2048
    bits = np.arange(0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(2)
    x = rng.choice(bits, size=t * hk * d).astype(np.uint16) | (rng.integers(0, 2, t * hk * d).astype(np.uint16) << 15)
    x = x.reshape(t, hk, d // 16, 16)
    # exponents of a block within 2^8 of one another, so that no code is trivially zero
    top = rng.integers(0x0800, 0x7F00, size=(t, hk, d // 16, 1)).astype(np.int64)
    x = ((x & 0x8000) | np.maximum(top - rng.integers(0, 0x500, size=x.shape), 0)).astype(np.uint16).reshape(t, hk, d)
    head = np.exp(rng.uniform(-60, 60, size=hk)).astype(np.float32)
    table = np.arange(t // 64, dtype=np.int32)[None]
    pool = np.zeros((t // 64, hk, 64 * (d // 2 + d // 16)), np.uint8)
    k, v = dev(pool), dev(pool)
    sh = ops.append_shapes(1, hk, d, t // 64, t // 64, t, "fp4")
    xb, h = ops.as_bf16(x, DEV), dev(head)
    ws = ops.append_kv(sh, xb, xb, dev(np.array([0, t], np.int32)), dev(np.zeros(1, np.int32)), dev(table), k, v, h, h)
    assert B.pa_check_status(ws) == B.PA_OK
    want = F.append(x, [0, t], [0], table, pool, head, d)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)


def test_zeros_keep_their_signs():
    d, hk = 64, 2
    x = W.bf16_normal(9, 0, (40, hk, d))
    x[:, :, 3::5] = 0x8000
    x[:, :, 1::7] = 0
    x[5:9, :, 2] = 0x8001  # rounds to -0
    x[9, 0, :16] = 0x8000  # nothing but zeros: codes 0
    head = np.array([0.37, 21.0], np.float32)
    table, pool = np.zeros((1, 1), np.int32), np.zeros((1, hk, 64 * (d // 2 + d // 16)), np.uint8)
    k, v, xb, h = dev(pool), dev(pool), ops.as_bf16(x, DEV), dev(head)
    ops.append_kv(ops.append_shapes(1, hk, d, 1, 1, 40, "fp4"), xb, xb, dev(np.array([0, 40], np.int32)),
                  dev(np.zeros(1, np.int32)), dev(table), k, v, h, h)
    want = F.append(x, [0, 40], [0], table, pool, head, d)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)


def gather_case(kv, d, hk, lens, start, seed=71):
    base = W.make_decode(len(lens), hk, hk, d, np.asarray(lens) + start, seed=seed, kv_dtype=kv, extra_pages=2)
    conv = {"bf16": ops.as_bf16, "f16": ops.as_f16, "e4m3": ops.as_e4m3}[kv]
    sc = (dev(base.k_scale), dev(base.v_scale)) if kv == "e4m3" else (None, None)
    def want(pool, scale):
        rows = []
        for b, n in enumerate(lens):
            for p in range(int(start[b]), int(start[b]) + n):
                r = pool[base.block_table[b, p // 64], :, p % 64]
                if kv == "e4m3":
                    r = W.f32_to_bf16_bits(oracle.e4m3_to_f64(np.ascontiguousarray(r)).astype(np.float32) * scale[:, None])
                rows.append(r)
        return np.stack(rows) if rows else np.zeros((0, hk, d), np.uint16)
    return base, conv(base.k_pool, DEV), conv(base.v_pool, DEV), sc, want(base.k_pool, base.k_scale), want(base.v_pool, base.v_scale)


@pytest.mark.parametrize("kv,d,hk", [("bf16", 128, 4), ("f16", 64, 3), ("e4m3", 128, 5), ("e4m3", 64, 9), ("bf16", 128, 1)])
def test_gather_bit_exact(kv, d, hk):
    lens, start = [1, 0, 65, 300, 64], np.array([0, 7, 63, 1, 128], np.int32)
    base, kp, vp, (ks, vs), kw, vw = gather_case(kv, d, hk, lens, start)
    cu = W.cu_seqlens(np.array(lens))
    pad = 3  # rows behind the last sequence stay as they were
    sh = ops.append_shapes(len(lens), hk, d, base.block_table.shape[1], base.num_pool_pages, int(cu[-1]) + pad, kv)
    dt = torch.float16 if kv == "f16" else torch.bfloat16
    ko, vo = (torch.full((sh.total_new, hk, d), 7.0, dtype=dt, device=DEV) for _ in range(2))
    _, _, ws = ops.gather_kv(sh, kp, vp, dev(cu), dev(start), dev(base.block_table), ks, vs, ko, vo)
    assert B.pa_check_status(ws) == B.PA_OK
    n = int(cu[-1])
    assert np.array_equal(ko[:n].view(torch.int16).cpu().numpy().view(np.uint16), kw)
    assert np.array_equal(vo[:n].view(torch.int16).cpu().numpy().view(np.uint16), vw)
    assert (ko[n:] == 7).all() and (vo[n:] == 7).all()


@pytest.mark.parametrize("d,hk", [(128, 4), (64, 5), (128, 1)])
def test_gather_fp4_bit_exact(d, hk):
    lens, start = np.array([1, 0, 65, 300], np.int32), np.array([0, 7, 63, 1], np.int32)
    c = Cache(lens + start, hk, d, seed=72)
    k, v, ks, vs, table, _ = c.up()
    cu = W.cu_seqlens(lens)
    sh = ops.append_shapes(len(lens), hk, d, c.table.shape[1], c.pages, int(cu[-1]), "fp4")
    ko, vo, ws = ops.gather_kv(sh, k, v, dev(cu), dev(start), table, ks, vs)
    assert B.pa_check_status(ws) == B.PA_OK
    for got, pool, head in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
        codes, scales = F.rows_of_slab(pool, d)
        rows = []
        for b in range(len(lens)):
            for p in range(int(start[b]), int(start[b] + lens[b])):
                page, r = c.table[b, p // 64], p % 64
                n = np.stack([codes[page, :, r] & 15, codes[page, :, r] >> 4], -1).reshape(hk, d).astype(int)
                val = (np.where(n >= 8, -1, 1) * F.GRID[n & 7]).astype(np.float32)
                step = oracle.e4m3_to_f64(np.ascontiguousarray(scales[page, :, r])).astype(np.float32) * head[:, None]
                rows.append(W.f32_to_bf16_bits(val * np.repeat(step, 16, -1)))
        bits = got.view(torch.int16).cpu().numpy().view(np.uint16)
        want = np.stack(rows)
        zero = (want & 0x7FFF) == 0  # -0 and +0 are one value
        assert np.array_equal(np.where(zero, 0, want), np.where((bits & 0x7FFF) == 0, 0, bits))


@pytest.mark.parametrize("kv", ["fp4", "bf16", "e4m3"])
def test_buffers_of_16_byte_alignment(kv):
    """Every buffer 16 bytes off a 32-byte boundary gives the bits of aligned ones."""
    d, hk, n = 64, 3, 150
    sc = (None, None) if kv == "bf16" else (torch.full((hk,), 0.02, device=DEV), torch.full((hk,), 0.03, device=DEV))

    def off(x):
        raw = torch.empty(x.numel() * x.element_size() + 16, dtype=torch.uint8, device=DEV)
        y = raw[16:].view(x.dtype).view(x.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(x)

    new = [ops.as_bf16(W.bf16_normal(74, s, (n, hk, d)), DEV) for s in (1, 2)]
    pools = [ops.kv_pool(3, hk, d, kv, DEV) for _ in range(2)]
    table, cu, start = dev(np.array([[2, 0, 1]], np.int32)), dev(np.array([0, n], np.int32)), dev(np.array([5], np.int32))
    sh = ops.append_shapes(1, hk, d, 3, 3, n, kv)
    got = []
    for wrap in (lambda x: x.clone(), off):
        kp, vp = wrap(pools[0]), wrap(pools[1])
        ws = ops.append_kv(sh, wrap(new[0]), wrap(new[1]), cu, start, table, kp, vp, *sc)
        ko, vo = wrap(torch.zeros_like(new[0])), wrap(torch.zeros_like(new[0]))
        ops.gather_kv(sh, kp, vp, cu, start, table, *sc, ko, vo, ws)
        assert B.pa_check_status(ws) == B.PA_OK
        got.append((kp.view(torch.uint8), vp.view(torch.uint8), ko, vo))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and got[0][2].any()


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_bad_pages_are_reported_and_skipped(kv):
    d, hk, n = 128, 4, 200
    shape = (5, hk, 64 * 72) if kv == "fp4" else (5, hk, 64, d)
    k = torch.zeros(shape, dtype=torch.uint8 if kv == "fp4" else torch.bfloat16, device=DEV)
    v, one = k.clone(), torch.ones(hk, device=DEV)
    sc = (one, one) if kv == "fp4" else (None, None)
    table = dev(np.array([[0, 9, -1, 3]], np.int32))  # pages 1 and 2 are bad ids
    new = torch.ones((n, hk, d), dtype=torch.bfloat16, device=DEV)
    cu, start = dev(np.array([0, n], np.int32)), dev(np.zeros(1, np.int32))
    sh = ops.append_shapes(1, hk, d, 4, 5, n, kv)
    ws = ops.append_kv(sh, new, new, cu, start, table, k, v, *sc)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    ko, vo = torch.full_like(new, 7), torch.full_like(new, 7)
    ops.gather_kv(sh, k, v, cu, start, table, *sc, ko, vo, ws)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    # a block of ones: its scale 1/6 lies nearest to 0.171875 of e4m3 (next to 0.15625), its code is 6
    back = 6 * 0.171875 if kv == "fp4" else 1.0
    for x in (ko, vo):
        assert (x[:64] == back).all() and (x[64:192] == 7).all() and (x[192:] == back).all()
    # a position past the block table
    ops.gather_kv(sh, k, v, cu, dev(np.array([100], np.int32)), dev(np.array([[0, 1, 2, 3]], np.int32)), *sc, ko, vo, ws)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    assert (ko[156:] == x[156:]).all()


def test_append_padding_is_not_read():
    d, hk = 64, 2
    c = Cache([10, 100], hk, d, seed=73, room=2)
    k, v, ks, vs, table, lens = c.up()
    new = W.bf16_normal(73, 92, (4, hk, d))
    cu = np.array([0, 1, 2], np.int32)  # two of the four tokens are padding
    ws = ops.append_kv(ops.append_shapes(2, hk, d, c.table.shape[1], c.pages, 4, "fp4"), ops.as_bf16(new, DEV),
                       ops.as_bf16(new, DEV), dev(cu), lens, table, k, v, ks, vs)
    assert B.pa_check_status(ws) == B.PA_OK
    assert np.array_equal(k.cpu().numpy(), F.append(new, cu, c.lens, c.table, c.k, c.ks, d))


# ----------------------------------------------------------------- attention

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 9, 16])
def test_decode_groups(d, group):
    c = Cache([1, 0, 63, 64, 65, 17, 300, 1000, 129], 2, d, seed=80 + group)
    c.poison()
    q, scale, out, lse, _ = decode(c, 2 * group, seed=group)
    check(c, q, scale, out, lse)


@pytest.mark.parametrize("n", list(range(1, 67)) + [127, 128, 255, 257, 511, 513])
def test_decode_every_short_length(n):
    c = Cache([n], 1, 128, seed=n)
    c.poison()
    q, scale, out, lse, _ = decode(c, 4, seed=n)
    check(c, q, scale, out, lse)


@pytest.mark.parametrize("forced,ctas", [(1, 1), (2, 0), (7, 2), (64, 4), (0, 1), (0, 8)])
def test_decode_splits(forced, ctas):
    c = Cache([5000, 1, 64, 777, 0, 4096], 3, 128, seed=90)
    c.poison()
    q, scale, out, lse, _ = decode(c, 12, forced_splits=forced, ctas_per_sm=ctas)
    check(c, q, scale, out, lse)


@pytest.mark.parametrize("scale,gain", [(3.0, 1.0), (-0.5, 1.0), (0.0, 1.0), (2.0 ** -30, 2.0 ** 20), (2.0 ** 20, 2.0 ** -30)])
def test_decode_scales(scale, gain):
    """Peaked, reversed and flat softmax; queries outside fp16's range."""
    c = Cache([700, 64], 2, 128, seed=91)
    q, scale, out, lse, _ = decode(c, 8, scale=scale, gain=gain)
    check(c, q, scale, out, lse)


def test_decode_growing_maximum():
    """Keys that grow along the sequence: the running maximum is raised all the way."""
    c = Cache([1500], 1, 128, seed=92)
    x = np.ones((c.pages, 1, 64, 128), np.float32)
    for i in range((1500 + 63) // 64):
        for r in range(64):
            x[c.table[0, i], 0, r] = (64 * i + r) / 1500 * 3
    c.k = F.make_pool(x, c.ks)
    q = W.f32_to_bf16_bits(np.full((1, 4, 128), 1.0, np.float32) * np.array([1, -1, 0.1, 8])[None, :, None].astype(np.float32))
    p = ops.plan_decode(c.lens, None, 4, 1, 128, c.table.shape[1], c.pages, kv_dtype="fp4")
    k, v, ks, vs, table, lens = c.up()
    out, lse = ops.decode(p, ops.as_bf16(q, DEV), k, v, table, lens, 0.3, ks, vs)
    assert B.pa_check_status(p.workspace) == B.PA_OK
    check(c, q, 0.3, out, lse)


def test_decode_nan_reaches_its_rows_only():
    c = Cache([200, 300], 2, 64, seed=93)
    codes, scales = F.rows_of_slab(c.k, 64)
    scales[c.table[0, 1], 1, 5] = 0x7F  # one key of sequence 0, KV head 1
    _, _, out, lse, _ = decode(c, 4)
    bad = torch.zeros((2, 4), dtype=torch.bool, device=DEV)
    bad[0, 2:] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(lse.isnan(), bad)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,hk,group,forced", [([4090, 70], 1, 8, 64), ([2000], 2, 3, 31),
                                                  ([4090, 300, 0, 64, 700, 513] + [50] * 120, 1, 15, 40)])
def test_merge_of_few_and_of_many_splits(d, lens, hk, group, forced):
    """Rows of up to 64 splits, alone or beside others: shared by the warps of a CTA, or a warp's own."""
    c = Cache(lens, hk, d, seed=95)
    q, scale, out, lse, p = decode(c, hk * group, forced_splits=forced)
    splits = [max(1, min(forced, 64, -(-n // 64))) if n > 64 else 1 for n in lens]
    assert p.plan.total_splits == sum(splits)
    check(c, q, scale, out, lse)


def test_attend_then_combine_and_noalloc():
    c = Cache([3000, 100, 0, 900], 2, 128, seed=94)
    q, scale, out, lse, p = decode(c, 8)
    k, v, ks, vs, table, lens = c.up()
    qd = ops.as_bf16(q, DEV)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    args = (p.shapes, p.plan, qd, k, v, ks, vs, table, lens, p.meta_dev, scale, o2, l2)
    B.pa_decode_attend(*args, p.workspace)
    B.pa_decode_combine(p.shapes, p.plan, p.meta_dev, o2, l2, p.workspace)
    assert B.pa_check_status(p.workspace) == B.PA_OK
    check(c, q, scale, o2, l2)
    o2.zero_()
    assert B.pa_decode_noalloc(*args) == B.PA_OK
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_decode_is_deterministic_and_batch_invariant_of_page_ids():
    c = Cache([3000, 100, 2000], 4, 128, seed=95)
    q, scale, out, lse, p = decode(c, 16)
    k, v, ks, vs, table, lens = c.up()
    for _ in range(5):
        o2, l2 = ops.decode(p, ops.as_bf16(q, DEV), k, v, table, lens, scale, ks, vs)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    perm = np.random.default_rng(0).permutation(c.pages)
    k2, v2 = np.empty_like(c.k), np.empty_like(c.v)
    k2[perm], v2[perm] = c.k, c.v
    o2, l2 = ops.decode(p, ops.as_bf16(q, DEV), dev(k2), dev(v2), dev(perm[c.table].astype(np.int32)), lens, scale, ks, vs)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert B.pa_check_status(p.workspace) == B.PA_OK


def test_decode_bad_page_and_long_length_are_reported():
    c = Cache([300, 200], 2, 128, seed=96)
    k, v, ks, vs, table, lens = c.up()
    p = ops.plan_decode(c.lens, None, 4, 2, 128, c.table.shape[1], c.pages, kv_dtype="fp4")
    q = ops.as_bf16(W.bf16_normal(96, 1, (2, 4, 128)), DEV)
    good, _ = ops.decode(p, q, k, v, table, lens, 0.1, ks, vs)
    assert B.pa_check_status(p.workspace) == B.PA_OK
    bad = table.clone()
    bad[0, 2] = c.pages
    out, _ = ops.decode(p, q, k, v, bad, lens, 0.1, ks, vs)
    assert B.pa_check_status(p.workspace) == B.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(out[1], good[1]) and out.isfinite().all()
    p.workspace.zero_()
    out, _ = ops.decode(p, q, k, v, table, torch.tensor([300, 2 ** 31 - 1], dtype=torch.int32, device=DEV), 0.1, ks, vs)
    assert B.pa_check_status(p.workspace) == B.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(out[0], good[0])


def test_decode_many_items_per_cta():
    """More work items than a CTA decodes ahead, most of them of one page."""
    lens = np.random.default_rng(7).integers(0, 100, size=700)
    c = Cache(lens, 2, 64, seed=97, extra=0)
    c.poison()
    q, scale, out, lse, _ = decode(c, 4, sms=2, ctas_per_sm=3)
    check(c, q, scale, out, lse)


@pytest.mark.parametrize("batch,longest,hk,sms", [(4, 32768, 8, 152), (20, 6000, 8, 152), (64, 4096, 1, 152),
                                                  (300, 500, 2, 152), (7, 900, 3, 5), (1, 70, 1, 1)])
def test_device_plan_is_the_host_plan(batch, longest, hk, sms):
    for seed in range(4):
        rng = np.random.default_rng(seed)
        lens = rng.integers(0, longest + 1, size=batch).astype(np.int32)
        if seed == 3:
            lens[:] = longest
        sh = B.pa_decode_shapes(batch=batch, num_q_heads=hk, num_kv_heads=hk, head_dim=128, page_size=64,
                                max_pages_per_seq=-(-longest // 64), num_pool_pages=1, kv_dtype=B.PA_KV_FP4_E2M1,
                                num_sms=sms, ctas_per_sm=0, forced_splits=0)
        host, _ = B.pa_get_metadata(lens, None, sh)
        plan = B.pa_get_static_plan(sh)
        meta = torch.zeros(plan.meta_ints, dtype=torch.int32, device=DEV)
        B.pa_get_metadata_device(sh, plan, dev(lens), meta)
        one, two = S.unpack(host.tolist()), S.unpack(meta.cpu().tolist())
        assert one["n_splits"] == two["n_splits"] and one["grid"] == two["grid"]
        assert sorted(one["items"]) == sorted(two["items"][:len(one["items"])])


def test_captured_step_follows_new_lengths():
    """append, device metadata and decode captured once and replayed as the sequences grow."""
    nb, hk, hq, d, steps = 5, 2, 8, 128, 3
    prior = np.array([0, 63, 200, 64, 900], np.int32)
    c = Cache(prior, hk, d, seed=98, room=steps)
    sh = B.pa_decode_shapes(batch=nb, num_q_heads=hq, num_kv_heads=hk, head_dim=d, page_size=64,
                            max_pages_per_seq=c.table.shape[1], num_pool_pages=c.pages, kv_dtype=B.PA_KV_FP4_E2M1,
                            num_sms=ops.num_sms(), ctas_per_sm=0, forced_splits=0)
    plan = B.pa_get_static_plan(sh)
    assert plan.ctas_per_sm == 3
    meta = torch.zeros(plan.meta_ints, dtype=torch.int32, device=DEV)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    aws = torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=DEV)
    k, v, ks, vs, table, start = c.up()
    lens = start + 1
    cu = torch.arange(nb + 1, dtype=torch.int32, device=DEV)
    kn, vn, q = (torch.zeros((nb, h, d), dtype=torch.bfloat16, device=DEV) for h in (hk, hk, hq))
    out = torch.empty_like(q)
    lse = torch.empty((nb, hq), device=DEV)
    ash = ops.append_shapes(nb, hk, d, c.table.shape[1], c.pages, nb, "fp4")

    def step():
        B.pa_append_kv(ash, kn, vn, cu, start, table, k, v, ks, vs, aws)
        B.pa_get_metadata_device(sh, plan, lens, meta)
        B.pa_decode(sh, plan, q, k, v, ks, vs, table, lens, meta, d ** -0.5, out, lse, ws)

    k0, v0 = k.clone(), v.clone()
    step()  # warm up outside the capture
    k.copy_(k0), v.copy_(v0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    k.copy_(k0), v.copy_(v0)
    for r in range(steps):
        bits = [W.bf16_normal(98, 10 * r + i, (nb, h, d)) for i, h in enumerate((hk, hk, hq))]
        for x, b in zip((kn, vn, q), bits):
            x.copy_(ops.as_bf16(b, DEV))
        g.replay()
        torch.cuda.synchronize()
        c.k = F.append(bits[0], np.arange(nb + 1), prior + r, c.table, c.k, c.ks, d)
        c.v = F.append(bits[1], np.arange(nb + 1), prior + r, c.table, c.v, c.vs, d)
        c.lens = prior + r + 1
        assert np.array_equal(k.cpu().numpy(), c.k)
        check(c, bits[2], d ** -0.5, out, lse)
        start += 1
        lens += 1
    assert B.pa_check_status(ws) == B.PA_OK and B.pa_check_status(aws) == B.PA_OK


def test_decode_without_lse_and_with_stale_workspace_contents():
    c = Cache([900, 10, 0], 2, 128, seed=101)
    q, scale, out, lse, p = decode(c, 8)
    k, v, ks, vs, table, lens = c.up()
    p.workspace[B.PA_STATUS_BYTES:].fill_(0xFF)  # partials are written before they are read
    o2 = torch.full_like(out, 7.0)
    B.pa_decode(p.shapes, p.plan, ops.as_bf16(q, DEV), k, v, ks, vs, table, lens, p.meta_dev, scale, o2, None, p.workspace)
    assert B.pa_check_status(p.workspace) == B.PA_OK
    assert torch.equal(o2, out)


def test_decode_of_a_grid_wider_than_its_items():
    """A capacity plan's launch: most CTAs have nothing to do, none of the sequences is split."""
    c = Cache([3, 200], 1, 64, seed=102)
    sh = B.pa_decode_shapes(batch=2, num_q_heads=3, num_kv_heads=1, head_dim=64, page_size=64,
                            max_pages_per_seq=c.table.shape[1], num_pool_pages=c.pages, kv_dtype=B.PA_KV_FP4_E2M1,
                            num_sms=ops.num_sms(), ctas_per_sm=0, forced_splits=0)
    plan = B.pa_get_static_plan(sh)
    meta = torch.zeros(plan.meta_ints, dtype=torch.int32, device=DEV)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    k, v, ks, vs, table, lens = c.up()
    q = W.bf16_normal(102, 1, (2, 3, 64))
    out, lse = torch.empty((2, 3, 64), dtype=torch.bfloat16, device=DEV), torch.empty((2, 3), device=DEV)
    B.pa_get_metadata_device(sh, plan, lens, meta)
    B.pa_decode(sh, plan, ops.as_bf16(q, DEV), k, v, ks, vs, table, lens, meta, 0.125, out, lse, ws)
    assert B.pa_check_status(ws) == B.PA_OK
    check(c, q, 0.125, out, lse)


def test_two_streams_with_their_own_workspaces():
    c = Cache([2000, 500], 2, 128, seed=99)
    k, v, ks, vs, table, lens = c.up()
    q = [ops.as_bf16(W.bf16_normal(99, s, (2, 8, 128)), DEV) for s in range(2)]
    plans = [ops.plan_decode(c.lens, None, 8, 2, 128, c.table.shape[1], c.pages, kv_dtype="fp4") for _ in range(2)]
    want = [ops.decode(plans[0], x, k, v, table, lens, 0.1, ks, vs) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(ops.decode(plans[i], q[i], k, v, table, lens, 0.1, ks, vs))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])


def test_chunk_through_the_cache_and_a_prefill():
    """A chunk over a 4-bit cache: append, read everything back, attend causally over it."""
    prefix, new = np.array([0, 70, 500], np.int32), np.array([40, 129, 256], np.int32)
    hq, hk, d = 8, 4, 128
    c = Cache(prefix, hk, d, seed=100, room=new)
    cu_q, cu_k = W.cu_seqlens(new), W.cu_seqlens(prefix + new)
    kn, vn, q = (W.bf16_normal(100, s, (int(cu_q[-1]), h, d)) for s, h in ((1, hk), (2, hk), (3, hq)))
    k, v, ks, vs, table, start = c.up()
    ws = ops.append_kv(ops.append_shapes(3, hk, d, c.table.shape[1], c.pages, int(cu_q[-1]), "fp4"),
                       ops.as_bf16(kn, DEV), ops.as_bf16(vn, DEV), dev(cu_q), start, table, k, v, ks, vs)
    kr, vr, _ = ops.gather_kv(ops.append_shapes(3, hk, d, c.table.shape[1], c.pages, int(cu_k[-1]), "fp4"), k, v,
                              dev(cu_k), dev(np.zeros(3, np.int32)), table, ks, vs, workspace=ws)
    sh = ops.prefill_shapes(3, hq, hk, d, d, 0, int(new.max()), int(cu_q[-1]), int(cu_k[-1]))
    out, lse, pws = ops.prefill(sh, ops.as_bf16(q, DEV), kr, vr, dev(cu_q), dev(cu_k), d ** -0.5, True)
    assert B.pa_check_status(ws) == B.PA_OK and B.pa_check_status(pws) == B.PA_OK
    bits = lambda x: x.view(torch.int16).cpu().numpy().view(np.uint16)
    ro, rl = oracle.prefill(q, bits(kr), bits(vr), cu_q, cu_k, d ** -0.5, True)
    err = np.abs(out.float().cpu().numpy() - ro)
    assert err.max() <= 1e-2 and err.mean() <= 1e-3 and np.abs(lse.cpu().numpy() - rl).max() <= 1e-3
    c.k, c.v = F.append(kn, cu_q, prefix, c.table, c.k, c.ks, d), F.append(vn, cu_q, prefix, c.table, c.v, c.vs, d)
    kv, _ = c.values()
    rows = np.concatenate([kv[c.table[b, :(n + 63) // 64]].transpose(0, 2, 1, 3).reshape(-1, hk, d)[:n]
                           for b, n in enumerate(prefix + new)])
    got = kr.float().cpu().numpy()
    assert (np.abs(got - rows) <= 2.0 ** -8 * np.abs(rows)).all()  # one bf16 rounding


@pytest.mark.parametrize("hq", [4, 8, 16])
@pytest.mark.parametrize("top", [1e3, 1e6, 1.3e7, 3e7, 6e7, 1e9, 1e12])
def test_decode_of_huge_logits_stays_finite(hq, top):
    """Logits whose fp32 steps are up to whole bits, the later pages' a few steps above the first ones': no weight
    overflows on the way, whichever way the steps round."""
    d, n = 128, 320
    j = [(a, b) for a in range(8) for b in (0, 2)]  # codes: step a's value, and 8 times b's
    c = Cache([n] * len(j), 1, d, seed=104)
    c.ks = c.vs = one = np.ones(1, np.float32)
    c.k, c.v = (F.make_pool(np.full((c.pages, 1, 64, d), 6, np.float32), one) for _ in range(2))
    codes, _ = F.rows_of_slab(c.k, d)  # scales are 1 throughout
    codes[:, 0, :, :8] = 0
    for i, (a, b) in enumerate(j):  # a warp's first page holds the first block's zeros, its second one the codes
        codes[c.table[i, 4], 0, :, 0] = a + 16 * b
    x = np.ones((len(j), hq, d), np.float32)
    x[..., 0], x[..., 1] = 2.0 ** -14, 2.0 ** -11  # 2^-14: an fp32 step of 672, the other blocks' product
    q = ops.as_bf16(W.f32_to_bf16_bits(x), DEV)
    p = ops.plan_decode(c.lens, None, hq, 1, d, c.table.shape[1], c.pages, kv_dtype="fp4", forced_splits=1)
    k, v, ks, vs, table, lens = c.up()
    for at in range(24):
        out, lse = ops.decode(p, q, k, v, table, lens, top * (1 + at / 37) / 672, ks, vs)
        assert B.pa_check_status(p.workspace) == B.PA_OK
        # every value is 6, so is every mean of them, but for P's fp16 (2^-11) and the output's bf16 rounding (2^-8),
        # and a few fp32 ones
        assert (out.float() - 6).abs().max() <= 6 * (2.0 ** -8 + 2.0 ** -10) and torch.isfinite(lse).all()


@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("bits", [20.0, 24.3, 27.7, 30.4])
def test_decode_of_many_keys_far_below_a_dominant_one(group, bits):
    """One key whose value row is zero, thousands of keys 2^-bits below it: what they weigh is the whole output, beside
    a sum that the dominant key makes."""
    d, n = 128, 4096
    c = Cache([n], 1, d, seed=103)
    c.ks = c.vs = one = np.ones(1, np.float32)
    # keys are 0 but for two blocks of key 0; values are 6 but for key 0's, which are 0
    x = np.zeros((c.pages, 1, 64, d), np.float32)
    x[c.table[0, 0], 0, 0, :32] = 6
    y = np.full((c.pages, 1, 64, d), 6, np.float32)
    y[c.table[0, 0], 0, 0] = 0
    c.k, c.v = F.make_pool(x, one), F.make_pool(y, one)
    kv, vv = c.values()
    assert np.array_equal(kv, x) and np.array_equal(vv, y)
    q = W.f32_to_bf16_bits(np.ones((1, group, d), np.float32))
    scale = float(np.float32(bits * np.log(2.0) / 192))  # the dominant logit: 192 scale, that is `bits` bits
    p = ops.plan_decode(c.lens, None, group, 1, d, c.table.shape[1], c.pages, kv_dtype="fp4", forced_splits=1)
    k, v, ks, vs, table, lens = c.up()
    out, lse = ops.decode(p, ops.as_bf16(q, DEV), k, v, table, lens, scale, ks, vs)
    assert B.pa_check_status(p.workspace) == B.PA_OK
    ro, rl, *_ = F.attend(q, kv, vv, c.table, c.lens, scale)
    # A weight lies within 2^-11 of itself, or 2^-32 of the largest where fp16 has no normal number for it: half a step
    # 2^-25 beside a largest weight of 2^7.  The logits' fp32 steps, at up to 31 bits, and the exponential's come to
    # less than 2^-17 relative.  The output is about 6 (n - 1) 2^-bits, and its bf16 rounding 2^-8 of it.
    tol = ro * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17) + 6 * n * 2.0 ** -32
    err = np.abs(out.double().cpu().numpy() - ro)
    assert (ro > 0).all() and (err <= tol).all(), float((err / ro).max())
    assert (np.abs(lse.cpu().numpy() - rl) <= 2.0 ** -19 * (1 + np.abs(rl))).all()


@pytest.mark.parametrize("d", [64, 128])
def test_combine_right_behind_the_device_metadata(d):
    """The merge called on its own, directly after the metadata was written on
    the device: it reads what was written, not what the buffer held before."""
    c = Cache([4000, 100, 0, 900, 3000], 2, d, seed=105)
    hq, nb = 16, len(c.lens)
    sh = B.pa_decode_shapes(batch=nb, num_q_heads=hq, num_kv_heads=2, head_dim=d, page_size=64,
                            max_pages_per_seq=c.table.shape[1], num_pool_pages=c.pages, kv_dtype=B.PA_KV_FP4_E2M1,
                            num_sms=ops.num_sms(), ctas_per_sm=0, forced_splits=0)
    plan = B.pa_get_static_plan(sh)
    meta = torch.zeros(plan.meta_ints, dtype=torch.int32, device=DEV)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    k, v, ks, vs, table, lens = c.up()
    q = W.bf16_normal(105, 1, (nb, hq, d))
    out, lse = torch.empty((nb, hq, d), dtype=torch.bfloat16, device=DEV), torch.empty((nb, hq), device=DEV)
    B.pa_get_metadata_device(sh, plan, lens, meta)
    B.pa_decode_attend(sh, plan, ops.as_bf16(q, DEV), k, v, ks, vs, table, lens, meta, d ** -0.5, out, lse, ws)
    splits = S.unpack(meta.cpu().tolist())["n_splits"]
    split = torch.tensor([n > 1 for n in splits], device=DEV)
    assert split.any() and not split.all()
    B.pa_decode_combine(sh, plan, meta, out, lse, ws)
    assert B.pa_check_status(ws) == B.PA_OK
    check(c, q, d ** -0.5, out, lse)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(50):
        meta.zero_()  # a merge that looked too early would find no splits
        o2.fill_(7.0)
        B.pa_get_metadata_device(sh, plan, lens, meta)
        B.pa_decode_combine(sh, plan, meta, o2, l2, ws)
        assert torch.equal(o2[split], out[split]) and torch.equal(l2[split], lse[split]) and (o2[~split] == 7).all()
    assert B.pa_check_status(ws) == B.PA_OK


@pytest.mark.parametrize("kv", ["fp4", "bf16", "e4m3"])
def test_gather_past_the_table_leaves_rows_as_they_were(kv):
    """Positions 100 .. 299 of a sequence whose block table has 256: the rows of 256 and beyond keep what they held,
    in the keys and in the values."""
    d, hk, n = 128, 2, 200
    sc = (None, None) if kv == "bf16" else (torch.full((hk,), 0.02, device=DEV), torch.full((hk,), 0.03, device=DEV))
    pools = [ops.kv_pool(5, hk, d, kv, DEV) for _ in range(2)]
    table = dev(np.array([[4, 1, 0, 3]], np.int32))
    new = [ops.as_bf16(W.bf16_normal(75, s, (256, hk, d)), DEV) for s in (1, 2)]
    cu = lambda m: dev(np.array([0, m], np.int32))
    zero = dev(np.zeros(1, np.int32))
    ws = ops.append_kv(ops.append_shapes(1, hk, d, 4, 5, 256, kv), *new, cu(256), zero, table, *pools, *sc)
    whole = ops.gather_kv(ops.append_shapes(1, hk, d, 4, 5, 256, kv), *pools, cu(256), zero, table, *sc, workspace=ws)[:2]
    assert B.pa_check_status(ws) == B.PA_OK
    out = [torch.full((n, hk, d), x, dtype=torch.bfloat16, device=DEV) for x in (7.0, 9.0)]
    ops.gather_kv(ops.append_shapes(1, hk, d, 4, 5, n, kv), *pools, cu(n), dev(np.array([100], np.int32)), table, *sc, *out, ws)
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    for got, want, x in zip(out, whole, (7.0, 9.0)):
        assert torch.equal(got[:156], want[100:]) and (got[156:] == x).all()
