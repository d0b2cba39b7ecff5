"""pa_qk_norm_rope against fp64, and pa_norm_rope_append_kv bit for bit
against pa_qk_norm_rope followed by pa_append_kv."""
import numpy as np
import pytest
import torch

from oracle import fp4 as F
from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops
from paged_kv_attention_fwd_gb300 import workloads as W
from paged_kv_attention_fwd_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(t, hq, hk, d, dtype, axes=1, rot=None, max_pos=4096, seed=0, packed=True, gain=1.0):
    rot = d if rot is None else rot
    g = torch.Generator().manual_seed(seed)
    qkv = (gain * torch.randn((t, (hq + 2 * hk) * d), generator=g)).to(TORCH[dtype]).to(DEV)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], -1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(TORCH[dtype]).to(DEV) for _ in range(2)]
    pos = torch.randint(0, max_pos, (axes, t), generator=g, dtype=torch.int32).to(DEV)
    cut = sorted(torch.randint(0, rot // 2 + 1, (axes - 1,), generator=g).tolist())
    sections = [b - a for a, b in zip([0] + cut, cut + [rot // 2])]
    return q, k, v, w, pos, sections, ops.rope_table(max_pos, rot, device=DEV) if rot else None


def compare(got, x, weight, pos, table, rot, inter, sections, eps, norm, dtype):
    f = lambda a: None if a is None else a.double().cpu().numpy()
    want, size = F.norm_rope(f(x), f(weight), pos.cpu().numpy(), table.cpu().numpy() if rot else None, rot, inter,
                             sections, eps, norm)
    # half a step of the type (2^-25 absolute below fp16's normal range), and the fp32 arithmetic: D / 2 roundings of
    # the sum of squares on the way to the norm (half of it after the square root) and 8 more
    d = x.shape[-1]
    tol = HALF_STEP[dtype] * np.abs(want) + (d / 4 + 8) * 2.0 ** -24 * size + (2.0 ** -25 if dtype == "f16" else 1e-40)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hk", [(1, 8, 2), (3, 1, 1), (5, 5, 3), (130, 16, 4), (1, 33, 7), (37, 32, 16)])
def test_against_fp64(d, dtype, inter, t, hq, hk):
    q, k, _, w, pos, sections, table = make(t, hq, hk, d, dtype, seed=t + d)
    sh = ops.rope_shapes(q, k, rope_dim=d, max_position=4096, interleaved=inter, sections=sections, eps=1e-6)
    qo, ko, ws = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table)
    assert B.pa_check_status(ws) == B.PA_OK
    compare(qo, q, w[0], pos, table, d, inter, sections, 1e-6, True, dtype)
    compare(ko, k, w[1], pos, table, d, inter, sections, 1e-6, True, dtype)


@pytest.mark.parametrize("rot", [0, 8, 24, 48, 64, 104, 128])
@pytest.mark.parametrize("axes", [1, 2, 3])
@pytest.mark.parametrize("inter", [False, True])
def test_partial_rotation_and_axes(rot, axes, inter):
    for seed in range(3):
        q, k, _, w, pos, sections, table = make(9, 6, 2, 128, "bf16", axes=axes, rot=rot, seed=seed)
        sh = ops.rope_shapes(q, k, rope_dim=rot, max_position=4096, interleaved=inter, sections=sections, eps=1e-5)
        qo, ko, ws = ops.qk_norm_rope(sh, q, k, w[0], None, pos, table)
        assert B.pa_check_status(ws) == B.PA_OK
        compare(qo, q, w[0], pos, table, rot, inter, sections, 1e-5, True, "bf16")
        compare(ko, k, None, pos, table, rot, inter, sections, 1e-5, True, "bf16")


def test_rotation_alone_in_place_and_queries_alone():
    q, k, v, w, pos, sections, table = make(77, 12, 4, 128, "f16", seed=5)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    sh = ops.rope_shapes(q, k, rope_dim=128, max_position=4096, norm=False, q_out=q, k_out=k)
    ops.qk_norm_rope(sh, q, k, None, None, pos, table, q_out=q, k_out=k)
    compare(q, q0, None, pos, table, 128, False, [64], 0, False, "f16")
    compare(k, k0, None, pos, table, 128, False, [64], 0, False, "f16")
    assert torch.equal(v, v0)  # the rest of the packed rows is untouched
    none = q[:, :0]
    sh = ops.rope_shapes(q0, none, rope_dim=128, max_position=4096, norm=False)
    qo, _, ws = ops.qk_norm_rope(sh, q0, none, None, None, pos, table)
    assert B.pa_check_status(ws) == B.PA_OK
    assert torch.equal(qo, q)


def test_zero_and_extreme_rows():
    q, k, _, w, pos, sections, table = make(6, 4, 2, 64, "bf16", seed=6)
    q = q.contiguous()
    q[0] = 0
    q[1] = 1e18
    q[2] = 1e-18
    q[3, 0, 5] = float("nan")
    sh = ops.rope_shapes(q, k, rope_dim=64, max_position=4096, eps=1e-6)
    qo, _, _ = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table)
    assert (qo[0] == 0).all()
    assert qo[3, 0].isnan().all() and qo[3, 1:].isfinite().all()
    keep = [1, 2, 4, 5]
    compare(qo[keep], q[keep], w[0], pos[:, keep], table, 64, False, [32], 1e-6, True, "bf16")


def test_padding_tokens_and_bad_positions():
    q, k, _, w, pos, sections, table = make(8, 4, 2, 128, "bf16", axes=2, seed=7)
    pos[0, 2] = -1       # padding
    pos[0, 5] = 4096     # past the table
    pos[1, 6] = -3       # a negative position of a later axis
    sh = ops.rope_shapes(q, k, rope_dim=128, max_position=4096, sections=sections)
    qo, ko = torch.full((8, 4, 128), 7.0, dtype=q.dtype, device=DEV), torch.full((8, 2, 128), 7.0, dtype=q.dtype, device=DEV)
    ws = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table, qo, ko)[2]
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    for i in (2, 5, 6):
        assert (qo[i] == 7).all() and (ko[i] == 7).all()
    keep = [0, 1, 3, 4, 7]
    compare(qo[keep], q[keep], w[0], pos[:, keep], table, 128, False, sections, 1e-6, True, "bf16")
    pos[0, 5], pos[1, 6] = 4095, 0
    ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table, qo, ko, ws)
    assert B.pa_check_status(ws) == B.PA_OK  # padding alone is no fault
    assert (qo[2] == 7).all()


@pytest.mark.parametrize("inter,axes,dtype", [(False, 1, "bf16"), (True, 3, "f16")])
def test_more_tokens_than_warps(inter, axes, dtype):
    """Every warp walks over several tokens, padding and bad positions among them."""
    q, k, _, w, pos, sections, table = make(7001, 6, 3, 64, dtype, axes=axes, rot=48, seed=11)
    pos[0, 5::97] = -1
    pos[-1, 11::301] = 4096
    sh = ops.rope_shapes(q, k, rope_dim=48, max_position=4096, interleaved=inter, sections=sections)
    qo, ko = (torch.full(x.shape, 7.0, dtype=x.dtype, device=DEV) for x in (q, k))
    ws = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table, qo, ko)[2]
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS
    skipped = ((pos < 0) | (pos >= 4096)).any(0)
    assert (qo[skipped] == 7).all() and (ko[skipped] == 7).all()
    keep = ~skipped
    compare(qo[keep], q[keep], w[0], pos[:, keep], table, 48, inter, sections, 1e-6, True, dtype)
    compare(ko[keep], k[keep], w[1], pos[:, keep], table, 48, inter, sections, 1e-6, True, dtype)


def test_keys_alone_and_no_rotation():
    q, k, _, w, _, _, _ = make(50, 4, 3, 128, "bf16", rot=0, seed=12)
    none = k[:, :0]
    sh = ops.rope_shapes(none, k, eps=1e-6)
    _, ko, ws = ops.qk_norm_rope(sh, none, k, None, w[1])
    assert B.pa_check_status(ws) == B.PA_OK
    compare(ko, k, w[1], torch.zeros((1, 50)), None, 0, False, [0], 1e-6, True, "bf16")


# ----------------------------------------------------------------- straight into the pages

@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3", "fp4"])
@pytest.mark.parametrize("d,hq,hk", [(128, 8, 2), (128, 5, 5), (64, 7, 1), (64, 16, 8), (128, 16, 8), (64, 16, 16)])
@pytest.mark.parametrize("inter,rot,axes", [(False, None, 1), (True, 40, 2), (False, 24, 3)])
def test_append_is_the_two_calls(kv, d, hq, hk, inter, rot, axes):
    dtype = "f16" if kv == "f16" else "bf16"
    prior, new = np.array([0, 63, 64, 130], np.int32), np.array([5, 1, 0, 70], np.int32)
    t = int(new.sum())
    q, k, v, w, pos, sections, table = make(t, hq, hk, d, dtype, axes=axes, rot=rot, seed=d + hq)
    bt, pages = W.assign_pages(prior + new, 3, 2)
    scales = [None, None] if kv in TORCH else [torch.full((hk,), s, device=DEV) for s in (0.011, 0.017)]
    one = [ops.kv_pool(pages, hk, d, kv, DEV) for _ in range(2)]
    two = [ops.kv_pool(pages, hk, d, kv, DEV) for _ in range(2)]
    cu, start, btd = dev(W.cu_seqlens(new)), dev(prior), dev(bt)
    ash = ops.append_shapes(4, hk, d, bt.shape[1], pages, t, kv)
    sh = ops.rope_shapes(q, k, v, rope_dim=d if rot is None else rot, max_position=4096, interleaved=inter,
                         sections=sections)
    qo, ko, ws = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table)
    ops.append_kv(ash, ko, v.contiguous(), cu, start, btd, *one, *scales, workspace=ws)
    q1, _ = ops.norm_rope_append_kv(sh, ash, q, k, v, cu, start, btd, *two, w[0], w[1], pos, table, *scales, workspace=ws)
    assert B.pa_check_status(ws) == B.PA_OK
    assert torch.equal(q1, qo)
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and a.view(torch.uint8).any()


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
@pytest.mark.parametrize("batch,longest", [(3, 3000), (126, 90), (127, 90), (128, 90), (300, 40), (2000, 4)])
def test_append_of_long_and_of_many_sequences(kv, batch, longest):
    """Warps that walk from sequence to sequence and from page to page, empty
    sequences among them, and batches past what one round of the search holds."""
    rng = np.random.default_rng(batch)
    new = rng.integers(0, longest + 1, size=batch).astype(np.int32)
    new[rng.integers(0, batch, size=1 + batch // 5)] = 0
    prior = rng.integers(0, 150, size=batch).astype(np.int32)
    d, hq, hk = 64, 6, 2
    t, pad = int(new.sum()), 5
    q, k, v, w, _, _, table = make(t + pad, hq, hk, d, "bf16", seed=batch)
    bt, pages = W.assign_pages(prior + new, batch, 2)
    scales = [None, None] if kv == "bf16" else [torch.full((hk,), s, device=DEV) for s in (0.011, 0.017)]
    one, two = ([ops.kv_pool(pages, hk, d, kv, DEV) for _ in range(2)] for _ in range(2))
    cu, start, btd = dev(W.cu_seqlens(new)), dev(prior), dev(bt)
    place = np.concatenate([prior[b] + np.arange(new[b]) for b in range(batch)] + [np.zeros(pad, int)]).astype(np.int32)
    ash = ops.append_shapes(batch, hk, d, bt.shape[1], pages, t + pad, kv)
    sh = ops.rope_shapes(q, k, v, rope_dim=d, max_position=4096)
    qo, ko, ws = ops.qk_norm_rope(sh, q, k, w[0], w[1], dev(place[None]), table)
    exact = ops.append_shapes(batch, hk, d, bt.shape[1], pages, t, kv)
    ops.append_kv(exact, ko[:t].contiguous(), v[:t].contiguous(), cu, start, btd, *one, *scales, workspace=ws)
    q1 = torch.full_like(qo, 7.0)
    ops.norm_rope_append_kv(sh, ash, q, k, v, cu, start, btd, *two, w[0], w[1], None, table, *scales, q_out=q1, workspace=ws)
    assert B.pa_check_status(ws) == B.PA_OK
    assert torch.equal(q1[:t], qo[:t]) and (q1[t:] == 7).all()
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # and back
    ko2, vo2, _ = ops.gather_kv(exact, *two, cu, start, btd, *scales, workspace=ws)
    if kv == "bf16":
        assert torch.equal(ko2, ko[:t]) and torch.equal(vo2, v[:t].contiguous())
    else:
        host = [x.cpu().numpy() for x in two]
        for got, pool, sc in zip((ko2, vo2), host, scales):
            val = F.decode_pool(pool, sc.cpu().numpy(), d)
            rows = np.concatenate([val[bt[b, p // 64], :, p % 64][None] for b in range(batch)
                                   for p in range(prior[b], prior[b] + new[b])])
            err = np.abs(got.double().cpu().numpy() - rows)
            assert (err <= 2.0 ** -8 * np.abs(rows)).all()  # one bf16 rounding
    assert B.pa_check_status(ws) == B.PA_OK


def test_append_positions_default_to_the_cache_and_padding_is_skipped():
    prior, new = np.array([10, 100], np.int32), np.array([3, 2], np.int32)
    q, k, v, w, _, _, table = make(8, 4, 2, 128, "bf16", seed=8)  # three padding tokens behind the last sequence
    bt, pages = W.assign_pages(prior + new, 4, 1)
    cu, start, btd = dev(W.cu_seqlens(new)), dev(prior), dev(bt)
    ash = ops.append_shapes(2, 2, 128, bt.shape[1], pages, 8)
    sh = ops.rope_shapes(q, k, v, rope_dim=128, max_position=4096)
    pos = torch.tensor([[10, 11, 12, 100, 101, 0, 0, 0]], dtype=torch.int32, device=DEV)
    pools = [[ops.kv_pool(pages, 2, 128, "bf16", DEV) for _ in range(2)] for _ in range(2)]
    outs = []
    for p, (kp, vp) in zip((pos, None), pools):
        qo = torch.full((8, 4, 128), 7.0, dtype=q.dtype, device=DEV)
        _, ws = ops.norm_rope_append_kv(sh, ash, q, k, v, cu, start, btd, kp, vp, w[0], w[1], p, table, q_out=qo)
        assert B.pa_check_status(ws) == B.PA_OK
        assert (qo[5:] == 7).all()
        outs.append(qo)
    assert torch.equal(outs[0], outs[1]) and torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    assert int((pools[0][1] != 0).any(-1).sum()) == 5 * 2  # five tokens' rows of two heads


@pytest.mark.parametrize("kv", ["e4m3", "fp4"])
@pytest.mark.parametrize("shuffled", [False, True])
def test_append_of_every_value_bit_for_bit(kv, shuffled):
    """Every bf16 bit pattern of a head, among neighbours of its size or of any, against scales of every size."""
    scales = torch.tensor([1.0, 0.37, 3.1e-3, 448.0, 7e-16, 2e15, 3e-30, 5e30], device=DEV)
    every = torch.arange(65536, dtype=torch.int32)
    if shuffled:
        every = every[torch.randperm(65536, generator=torch.Generator().manual_seed(3))]
    v = every.to(torch.int16).view(torch.bfloat16).view(512, 1, 128).expand(512, 8, 128).contiguous().to(DEV)
    bt = np.random.default_rng(4).permutation(9)[None].astype(np.int32)
    cu, start, btd = dev(np.array([0, 512], np.int32)), dev(np.array([33], np.int32)), dev(bt)
    ash = ops.append_shapes(1, 8, 128, 9, 9, 512, kv)
    pools = [ops.kv_pool(9, 8, 128, kv, DEV) for _ in range(4)]
    ops.append_kv(ash, v, v, cu, start, btd, pools[0], pools[1], scales, scales)
    sh = ops.rope_shapes(v, v, v, norm=False)  # a key that neither turns nor is normed passes through but for NaN's bits
    ops.norm_rope_append_kv(sh, ash, torch.zeros_like(v), v, v, cu, start, btd, pools[2], pools[3], k_scale=scales,
                            v_scale=scales)
    as_bytes = [p.view(torch.uint8) for p in pools]
    assert torch.equal(as_bytes[1], as_bytes[3]) and torch.equal(as_bytes[0], as_bytes[2])


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
@pytest.mark.parametrize("rot", [0, 64])
def test_append_in_place_and_without_rotation(kv, rot):
    """Queries written over the packed projection they came from; without a rotation positions are not looked at."""
    prior, new = np.array([60, 0, 7], np.int32), np.array([9, 1, 130], np.int32)
    q, k, v, w, pos, _, table = make(140, 6, 2, 64, "bf16", rot=rot, seed=10)
    bt, pages = W.assign_pages(prior + new, 4, 1)
    cu, start, btd = dev(W.cu_seqlens(new)), dev(prior), dev(bt)
    ash = ops.append_shapes(3, 2, 64, bt.shape[1], pages, 140, kv)
    scale = torch.full((2,), 0.37, device=DEV) if kv == "fp4" else None
    if rot == 0:
        pos = torch.full_like(pos, -1)
    runs = []
    for out in (torch.empty_like(q), q):
        kp, vp = (ops.kv_pool(pages, 2, 64, kv, DEV) for _ in range(2))
        sh = ops.rope_shapes(q, k, v, rope_dim=rot, max_position=4096, q_out=out)
        k0, v0 = k.clone(), v.clone()
        _, ws = ops.norm_rope_append_kv(sh, ash, q, k, v, cu, start, btd, kp, vp, w[0], w[1], pos, table, scale, scale,
                                        q_out=out)
        assert B.pa_check_status(ws) == B.PA_OK
        assert torch.equal(k, k0) and torch.equal(v, v0)
        runs.append((out, kp, vp))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert (runs[0][0] != 0).any(-1).all()


def test_append_reports_what_is_out_of_range():
    q, k, v, w, _, _, table = make(4, 4, 2, 64, "bf16", seed=9)
    bt = np.array([[0, 5]], np.int32)  # page id 5 of a pool of 2
    cu, btd = dev(np.array([0, 4], np.int32)), dev(bt)
    ash = ops.append_shapes(1, 2, 64, 2, 2, 4)
    sh = ops.rope_shapes(q, k, v, rope_dim=64, max_position=4096)
    for first, ok in ((0, 4), (62, 2), (126, 0), (-1, 3)):
        kp, vp = ops.kv_pool(2, 2, 64, "bf16", DEV), ops.kv_pool(2, 2, 64, "bf16", DEV)
        qo = torch.full((4, 4, 64), 7.0, dtype=q.dtype, device=DEV)
        _, ws = ops.norm_rope_append_kv(sh, ash, q, k, v, cu, dev(np.array([first], np.int32)), btd, kp, vp, w[0], w[1],
                                        None, table, q_out=qo)
        assert B.pa_check_status(ws) == (B.PA_OK if ok == 4 else B.PA_ERR_DEVICE_BOUNDS)
        assert int((qo != 7).any(-1).all(-1).sum()) == ok
        assert int((vp != 0).any(-1).sum()) == 2 * ok


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_whole_decode_steps(kv):
    """Steps as a serving loop issues them: norm, rotation and append in one
    call, then attention, on one stream without synchronisation; captured once
    and replayed as the sequences grow."""
    nb, hq, hk, d, steps = 6, 8, 2, 128, 3
    prior = np.array([0, 63, 64, 300, 1000, 5], np.int32)
    bt, pages = W.assign_pages(prior + steps, 5, 2)
    rng = np.random.default_rng(10)
    scales = np.array([0.012, 0.009], np.float32)
    sc = [dev(scales), dev(scales)] if kv == "fp4" else [None, None]
    kp, vp = ops.kv_pool(pages, hk, d, kv, DEV), ops.kv_pool(pages, hk, d, kv, DEV)
    host = [F.make_pool(rng.standard_normal((pages, hk, 64, d)).astype(np.float32), scales) if kv == "fp4"
            else W.f32_to_bf16_bits(rng.standard_normal((pages, hk, 64, d)).astype(np.float32)) for _ in range(2)]
    put = (lambda x: dev(x)) if kv == "fp4" else (lambda x: ops.as_bf16(x, DEV))
    qkv = torch.zeros((nb, (hq + 2 * hk) * d), dtype=torch.bfloat16, device=DEV)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], -1))
    w = [(1 + 0.1 * torch.randn(d)).to(torch.bfloat16).to(DEV) for _ in range(2)]
    table = ops.rope_table(2048, d, device=DEV)
    start, lens, btd = dev(prior), dev(prior + 1), dev(bt)
    cu = torch.arange(nb + 1, dtype=torch.int32, device=DEV)
    ash = ops.append_shapes(nb, hk, d, bt.shape[1], pages, nb, kv)
    sh = ops.rope_shapes(q, k, v, rope_dim=d, max_position=2048)
    dsh = B.pa_decode_shapes(batch=nb, num_q_heads=hq, num_kv_heads=hk, head_dim=d, page_size=64,
                             max_pages_per_seq=bt.shape[1], num_pool_pages=pages, kv_dtype=ops.KV_DTYPES[kv],
                             num_sms=ops.num_sms(), ctas_per_sm=0, forced_splits=0)
    plan = B.pa_get_static_plan(dsh)
    meta = torch.zeros(plan.meta_ints, dtype=torch.int32, device=DEV)
    ws, rws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
    qo, out = torch.empty((nb, hq, d), dtype=torch.bfloat16, device=DEV), torch.empty((nb, hq, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((nb, hq), device=DEV)

    def step():
        B.pa_norm_rope_append_kv(sh, ash, q, k, v, w[0], w[1], None, table, cu, start, btd, qo, kp, vp, *sc, rws)
        B.pa_get_metadata_device(dsh, plan, lens, meta)
        B.pa_decode(dsh, plan, qo, kp, vp, *sc, btd, lens, meta, d ** -0.5, out, lse, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kp.copy_(put(host[0])), vp.copy_(put(host[1]))
    for r in range(steps):
        qkv.copy_(torch.from_numpy(rng.standard_normal(tuple(qkv.shape)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        pos = (prior + r)[None]
        compare(qo, q, w[0], torch.from_numpy(pos), table, d, False, [d // 2], 1e-6, True, "bf16")
        bits = lambda x: np.ascontiguousarray(x.view(torch.uint8 if kv == "fp4" else torch.int16).cpu().numpy())
        kb, vb = bits(kp), bits(vp)
        if kv == "fp4":
            kf, vf = F.decode_pool(kb, scales, d), F.decode_pool(vb, scales, d)
        else:
            kf, vf = F.to_f64(kb.view(np.uint16), "bf16"), F.to_f64(vb.view(np.uint16), "bf16")
        ro, rl, *_ = F.attend(qo.view(torch.int16).cpu().numpy().view(np.uint16), kf, vf, bt, prior + r + 1, d ** -0.5)
        assert np.abs(out.float().cpu().numpy() - ro).max() <= 1e-2
        assert np.abs(lse.cpu().numpy() - rl).max() <= 1e-3
        for b in range(nb):  # the new token's row is the turned key, in the cache's precision
            p = int(prior[b]) + r
            want, _ = F.norm_rope(k[b:b + 1].double().cpu().numpy(), w[1].double().cpu().numpy(), pos[:, b:b + 1],
                                  table.cpu().numpy(), d, False, [d // 2], 1e-6)
            got = kf[bt[b, p // 64], :, p % 64]
            top = np.abs(want[0]).reshape(hk, -1, 16).max(-1).repeat(16, -1)
            # 4 bits: half the widest gap of the grid (1 of 6) of the block's largest, its scale 2^-4 off
            assert (np.abs(got - want[0]) <= (top / 6 * 1.0625 if kv == "fp4" else 2.0 ** -7 * np.abs(want[0]) + 1e-6)).all()
        start += 1
        lens += 1
    assert B.pa_check_status(ws) == B.PA_OK and B.pa_check_status(rws) == B.PA_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("axes", [1, 2])
def test_append_padding_by_position_wherever_the_token_lies(kv, axes):
    """Idle slots of a fixed batch: a token with a negative axis-0 position
    inside its sequence's range is padding, whatever its place in the cache
    is -- valid, an unset page id, or past the block table."""
    d, hq, hk, pages = 64, 5, 2, 4
    start = np.array([7, 70, 5, 500, 130], np.int32)   # the third's page id is unset, the fourth lies past the table
    bt = np.array([[0, -1], [1, 2], [-1, 2 ** 31 - 1], [3, 3], [-1, -1]], np.int32)
    q, k, v, w, pos, sections, table = make(5, hq, hk, d, "bf16", axes=axes, seed=13)
    idle = [1, 2, 3, 4]
    pos[0, idle] = torch.tensor([-1, -1, -5, -2 ** 31], dtype=torch.int32, device=DEV)
    scales = [None, None] if kv == "bf16" else [torch.full((hk,), s, device=DEV) for s in (0.011, 0.017)]
    kp, vp = (ops.kv_pool(pages, hk, d, kv, DEV) for _ in range(2))
    qo = torch.full((5, hq, d), 7.0, dtype=q.dtype, device=DEV)
    sh = ops.rope_shapes(q, k, v, rope_dim=d, max_position=4096, sections=sections)
    _, ws = ops.norm_rope_append_kv(sh, ops.append_shapes(5, hk, d, 2, pages, 5, kv), q, k, v,
                                    dev(np.arange(6, dtype=np.int32)), dev(start), dev(bt), kp, vp, w[0], w[1], pos, table,
                                    *scales, q_out=qo)
    assert B.pa_check_status(ws) == B.PA_OK
    assert (qo[idle] == 7).all() and (qo[0] != 7).any()
    assert not kp[1:].view(torch.uint8).any() and not vp[1:].view(torch.uint8).any()
    assert kp[0].view(torch.uint8).any() and vp[0].view(torch.uint8).any()
    compare(qo[:1], q[:1], w[0], pos[:, :1], table, d, False, sections, 1e-6, True, "bf16")


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3", "fp4"])
def test_append_padding_is_the_two_calls(kv):
    """Tokens behind the last sequence (and before the first) are padding in every form of the append and for every
    page type: nothing of them is written."""
    dtype = "f16" if kv == "f16" else "bf16"
    prior, new = np.array([10, 100, 3], np.int32), np.array([3, 40, 0], np.int32)
    d, hq, hk, lead, pad = 64, 3, 2, 2, 25
    t = lead + int(new.sum()) + pad
    q, k, v, w, pos, _, table = make(t, hq, hk, d, dtype, seed=14)
    bt, pages = W.assign_pages(prior + new + 64, 4, 1)   # room for the padding behind the last sequence
    scales = [None, None] if kv in TORCH else [torch.full((hk,), s, device=DEV) for s in (0.011, 0.017)]
    one, two, bare = ([ops.kv_pool(pages, hk, d, kv, DEV) for _ in range(2)] for _ in range(3))
    cu, start, btd = dev(lead + W.cu_seqlens(new)), dev(prior), dev(bt)
    ash = ops.append_shapes(3, hk, d, bt.shape[1], pages, t, kv)
    sh = ops.rope_shapes(q, k, v, rope_dim=d, max_position=4096)
    qo, ko, ws = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table)
    ops.append_kv(ash, ko, v.contiguous(), cu, start, btd, *one, *scales, workspace=ws)
    q1 = torch.full_like(qo, 7.0)
    ops.norm_rope_append_kv(sh, ash, q, k, v, cu, start, btd, *two, w[0], w[1], pos, table, *scales, q_out=q1, workspace=ws)
    live = slice(lead, t - pad)
    exact = ops.append_shapes(3, hk, d, bt.shape[1], pages, t - lead - pad, kv)
    ops.append_kv(exact, ko[live].contiguous(), v[live].contiguous(), cu - lead, start, btd, *bare, *scales, workspace=ws)
    assert B.pa_check_status(ws) == B.PA_OK
    assert torch.equal(q1[live], qo[live]) and (q1[:lead] == 7).all() and (q1[t - pad:] == 7).all()
    for a, b, c in zip(one, two, bare):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
        assert torch.equal(b.view(torch.uint8), c.view(torch.uint8)) and c.view(torch.uint8).any()


@pytest.mark.parametrize("call", ["append", "gather", "rope", "fused"])
@pytest.mark.parametrize("handle", [False, True])
def test_buffers_that_a_call_makes_belong_to_its_stream(call, handle):
    """A call on a stream of its own while the current one is busy: the status word that it makes is cleared before the
    kernel records its fault in it, not by a fill that the current stream comes to later."""
    t, d, hk = 6, 64, 2
    q, k, v, w, pos, _, table = make(t, 4, hk, d, "bf16", seed=15, packed=False)
    pos[0, 3] = 4096  # past the table
    pools = [ops.kv_pool(3, hk, d, "bf16", DEV) for _ in range(2)]
    cu, start, bt = dev(np.array([0, t], np.int32)), dev(np.array([60], np.int32)), dev(np.array([[1, 9]], np.int32))
    ash, sh = ops.append_shapes(1, hk, d, 2, 3, t), ops.rope_shapes(q, k, v, rope_dim=d, max_position=4096)
    busy = torch.zeros(1 << 28, device=DEV)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side

    def run():
        if call == "append":
            return ops.append_kv(ash, k, v, cu, start, bt, *pools, stream=stream)
        if call == "gather":
            return ops.gather_kv(ash, *pools, cu, start, bt, stream=stream)[2]
        if call == "rope":
            return ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table, stream=stream)[2]
        return ops.norm_rope_append_kv(sh, ash, q, k, v, cu, start, bt, *pools, w[0], w[1], None, table, stream=stream)[1]

    run()  # kernels are loaded at their first launch, which waits for the device
    busy.add_(1)
    torch.cuda.synchronize()
    for _ in range(40):
        busy.add_(1)
    ws = run()
    torch.cuda.synchronize()
    assert B.pa_check_status(ws) == B.PA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("stream", [0, 1, 2, "object"])
def test_streams_by_other_names(stream):
    """CUDA's handles of the default streams, and any object with a handle: the call makes its buffers and runs."""
    q, k, _, w, pos, _, table = make(5, 4, 2, 64, "bf16", seed=16)
    sh = ops.rope_shapes(q, k, rope_dim=64, max_position=4096)
    want = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Named:
        cuda_stream = side.cuda_stream

    got = ops.qk_norm_rope(sh, q, k, w[0], w[1], pos, table, stream=Named() if stream == "object" else stream)
    torch.cuda.synchronize()
    assert B.pa_check_status(got[2]) == B.PA_OK and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
