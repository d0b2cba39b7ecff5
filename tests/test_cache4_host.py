"""Host-side checks of the 4-bit page type, the read-back and the norm with
rotation: bad arguments are refused with the documented status before
anything is enqueued (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import scheduler as S
from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops
from paged_kv_attention_fwd_gb300.build import build

from .test_abi import _Fake, _decode_call, shapes


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def test_slab_bytes():
    assert [B.pa_page_slab_bytes(128, t) for t in range(4)] == [16384, 8192, 16384, 4608]
    assert [B.pa_page_slab_bytes(64, t) for t in range(4)] == [8192, 4096, 8192, 2304]
    assert B.pa_page_slab_bytes(96, 3) == 0 and B.pa_page_slab_bytes(128, 4) == 0


def plain_plan(lens, hk, cap, forced):
    """(splits per sequence, items of each CTA) of the 4-bit rule: one item per CTA share, and chunks up to 12 pages
    longer where that leaves no CTA with two."""
    pages = [-(-n // 64) for n in lens]
    chunk = max(4, -(-sum(pages) * hk // cap))
    one_each = [c for c in range(chunk, chunk + 13) if sum(max(1, min(64, -(-p // c))) for p in pages) * hk <= cap]
    chunk = one_each[0] if one_each else chunk
    n = [1 if p <= 1 else min(forced, p, 64) if forced else min(-(-p // chunk), 64) for p in pages]
    items = [((s + 1) * p // k - s * p // k + 1, b, s, g) for b, (p, k) in enumerate(zip(pages, n)) for s in range(k)
             for g in range(hk)]
    ctas = [[] for _ in range(min(len(items), cap))]
    loads = [[0, c] for c in range(len(ctas))]
    for cost, b, s, g in sorted(items, key=lambda i: -i[0]):  # stable: ties keep their order
        least = min(loads)
        least[0] += cost
        ctas[least[1]].append((b, s, g))
    return n, ctas


@pytest.mark.parametrize("lens,hq,forced", [([10, 3000, 0, 777], 32, 0), ([5000], 32, 0), ([4096] * 9, 128, 0),
                                            (list(range(0, 4000, 130)), 32, 0), ([640, 1000], 64, 5),
                                            ([2500], 32, 0), ([900, 1000], 32, 0), ([5120, 64], 128, 0)])
def test_plan_of_4_bit_pages(lens, hq, forced):
    for cps, want in ((0, 2 if hq > 64 else 3), (1, 1), (5, 5)):
        sh = shapes(len(lens), hq=hq, max_pages=80, sms=7, cps=cps, forced=forced, kv=B.PA_KV_FP4_E2M1)
        meta, plan = B.pa_get_metadata(np.array(lens, np.int32), None, sh)
        u = S.unpack(meta.tolist())
        n, ctas = plain_plan(lens, 8, 7 * want, forced)
        assert plan.ctas_per_sm == u["ctas_per_sm"] == want and u["n_splits"] == n and u["grid"] == len(ctas)
        ptr = u["cta_indptr"]
        assert [u["items"][ptr[c]:ptr[c + 1]] for c in range(len(ctas))] == ctas
        static = B.pa_get_static_plan(sh)
        assert static.total_splits >= u["total_splits"] and static.grid >= u["grid"]
        assert static.meta_ints >= plan.meta_ints and static.workspace_bytes >= plan.workspace_bytes
    assert B.pa_get_static_plan(shapes(4, cps=0)).ctas_per_sm == 1


@pytest.mark.parametrize("over,status,needle", [
    ({}, B.PA_ERR_INVALID_ARG, "k_scale"),
    ({"k_scale": _Fake()}, B.PA_ERR_INVALID_ARG, "4-bit"),
    ({"k_scale": _Fake(), "v_scale": _Fake(), "k_pool": _Fake(addr=(1 << 20) + 8)}, B.PA_ERR_INVALID_ARG, "aligned"),
])
def test_decode_refusals(over, status, needle):
    sh = shapes(2, kv=B.PA_KV_FP4_E2M1)
    _, plan = B.pa_get_metadata(np.array([100, 300], np.int32), None, sh)
    with pytest.raises(B.PaError) as e:
        _decode_call(sh, plan, **over)
    assert e.value.status == status and needle in str(e.value)


def test_unknown_page_type_is_refused():
    sh = shapes(2, kv=4)
    _, plan = B.pa_get_metadata(np.array([100, 300], np.int32), None, sh)
    with pytest.raises(B.PaError, match="kv_dtype"):
        _decode_call(sh, plan)


def test_mixed_batches_refuse_4_bit_pools():
    sh = B.pa_mixed_shapes(batch=1, num_q_heads=8, num_kv_heads=8, head_dim=128, page_size=64, max_pages_per_seq=4,
                           num_pool_pages=9, kv_dtype=B.PA_KV_FP4_E2M1, num_sms=152, ctas_per_sm=0, forced_splits=0)
    with pytest.raises(B.PaError) as e:
        B.pa_get_mixed_plan(np.array([0, 1], np.int32), np.array([5], np.int32), None, sh)
    assert e.value.status == B.PA_ERR_UNSUPPORTED


def cache_call(name, sh, **over):
    f = _Fake()
    a = dict(k_rows=f, v_rows=f, cu=f, start=f, table=f, k_pool=f, v_pool=f, k_scale=f, v_scale=f, ws=f)
    a.update(over)
    if name == "append":
        B.pa_append_kv(sh, a["k_rows"], a["v_rows"], a["cu"], a["start"], a["table"], a["k_pool"], a["v_pool"],
                       a["k_scale"], a["v_scale"], a["ws"], stream=1)
    else:
        B.pa_gather_kv(sh, a["k_pool"], a["v_pool"], a["k_scale"], a["v_scale"], a["cu"], a["start"], a["table"],
                       a["k_rows"], a["v_rows"], a["ws"], stream=1)


@pytest.mark.parametrize("name", ["append", "gather"])
@pytest.mark.parametrize("change,over,status,needle", [
    ({"kv_dtype": 4}, {}, B.PA_ERR_INVALID_ARG, "kv_dtype"),
    ({"head_dim": 96}, {}, B.PA_ERR_UNSUPPORTED, "head_dim"),
    ({"page_size": 16}, {}, B.PA_ERR_INVALID_ARG, "page_size"),
    ({"num_kv_heads": 0}, {}, B.PA_ERR_INVALID_ARG, "num_kv_heads"),
    ({"num_pool_pages": 0}, {}, B.PA_ERR_INVALID_ARG, "num_pool_pages"),
    ({"total_new": -1}, {}, B.PA_ERR_INVALID_ARG, "total_new"),
    ({}, {"k_scale": None}, B.PA_ERR_INVALID_ARG, "4-bit"),
    ({"kv_dtype": 1}, {"v_scale": None}, B.PA_ERR_INVALID_ARG, "e4m3"),
    ({}, {"table": None}, B.PA_ERR_INVALID_ARG, "NULL"),
    ({}, {"v_rows": _Fake(addr=(1 << 20) + 2)}, B.PA_ERR_INVALID_ARG, "aligned"),
    ({}, {"ws": _Fake(n=100)}, B.PA_ERR_WORKSPACE, "workspace"),
])
def test_cache_refusals(name, change, over, status, needle):
    sh = ops.append_shapes(2, 4, 128, 4, 9, 10, "fp4")
    for k, v in change.items():
        setattr(sh, k, v)
    with pytest.raises(B.PaError) as e:
        cache_call(name, sh, **over)
    assert e.value.status == status and needle in str(e.value)


def test_empty_cache_calls_do_nothing():
    for name in ("append", "gather"):
        cache_call(name, ops.append_shapes(0, 4, 128, 4, 9, 10, "fp4"), k_rows=None)
        cache_call(name, ops.append_shapes(3, 4, 128, 4, 9, 0, "fp4"), k_rows=None)


def rope(**change):
    sh = B.pa_rope_shapes(total_tokens=3, num_q_heads=8, num_kv_heads=2, head_dim=128, rope_dim=128, interleaved=0,
                          num_axes=2, max_position=100, dtype=B.PA_KV_BF16, norm=1, eps=1e-6, q_stride=1536,
                          k_stride=1536, v_stride=1536, q_out_stride=1024, k_out_stride=256)
    sh.sections[0], sh.sections[1] = 40, 24
    for k, v in change.items():
        if k == "sections":
            for i in range(3):
                sh.sections[i] = v[i]
        else:
            setattr(sh, k, v)
    return sh


def rope_call(sh, **over):
    f = _Fake()
    a = dict(q=f, k=f, qw=None, kw=None, pos=f, cs=f, qo=f, ko=f, ws=f)
    a.update(over)
    B.pa_qk_norm_rope(sh, *(a[n] for n in ("q", "k", "qw", "kw", "pos", "cs", "qo", "ko", "ws")), stream=1)


ROPE_REFUSALS = [
    ({"head_dim": 96}, {}, B.PA_ERR_UNSUPPORTED, "head_dim"),
    ({"dtype": 1}, {}, B.PA_ERR_INVALID_ARG, "dtype"),
    ({"rope_dim": 130}, {}, B.PA_ERR_INVALID_ARG, "rope_dim"),
    ({"rope_dim": 60}, {}, B.PA_ERR_INVALID_ARG, "rope_dim"),
    ({"num_axes": 4}, {}, B.PA_ERR_INVALID_ARG, "num_axes"),
    ({"sections": (40, 23, 0)}, {}, B.PA_ERR_INVALID_ARG, "pairs"),
    ({"sections": (40, 20, 4)}, {}, B.PA_ERR_INVALID_ARG, "sections[2]"),
    ({"sections": (65, -1, 0)}, {}, B.PA_ERR_INVALID_ARG, "sections[1]"),
    ({"max_position": 0}, {}, B.PA_ERR_INVALID_ARG, "max_position"),
    ({"norm": 2}, {}, B.PA_ERR_INVALID_ARG, "norm"),
    ({"eps": -1.0}, {}, B.PA_ERR_INVALID_ARG, "eps"),
    ({"eps": float("nan")}, {}, B.PA_ERR_INVALID_ARG, "eps"),
    ({"q_stride": 1000}, {}, B.PA_ERR_INVALID_ARG, "q_stride"),
    ({"q_stride": 1540}, {}, B.PA_ERR_INVALID_ARG, "q_stride"),
    ({"num_q_heads": 0, "num_kv_heads": 0}, {}, B.PA_ERR_INVALID_ARG, "num_q_heads"),
    ({"total_tokens": -1}, {}, B.PA_ERR_INVALID_ARG, "total_tokens"),
    ({}, {"q": None}, B.PA_ERR_INVALID_ARG, "NULL"),
    ({}, {"cs": None}, B.PA_ERR_INVALID_ARG, "NULL"),
    ({}, {"kw": _Fake(addr=(1 << 20) + 4)}, B.PA_ERR_INVALID_ARG, "aligned"),
    ({}, {"ws": _Fake(n=8)}, B.PA_ERR_WORKSPACE, "workspace"),
]


@pytest.mark.parametrize("change,over,status,needle", ROPE_REFUSALS + [
    ({"k_out_stride": 8}, {}, B.PA_ERR_INVALID_ARG, "k_out_stride"),
    ({}, {"pos": None}, B.PA_ERR_INVALID_ARG, "NULL"),
    ({}, {"ko": None}, B.PA_ERR_INVALID_ARG, "NULL"),
    ({}, {"ko": _Fake(addr=(1 << 20) + 4)}, B.PA_ERR_INVALID_ARG, "aligned"),
])
def test_norm_rope_refusals(change, over, status, needle):
    with pytest.raises(B.PaError) as e:
        rope_call(rope(**change), **over)
    assert e.value.status == status and needle in str(e.value)


def fused_call(sh, ap, **over):
    f = _Fake()
    a = dict(q=f, k=f, v=f, qw=None, kw=None, pos=f, cs=f, cu=f, start=f, table=f, qo=f, kp=f, vp=f, ks=None, vs=None, ws=f)
    a.update(over)
    B.pa_norm_rope_append_kv(sh, ap, *a.values(), stream=1)


@pytest.mark.parametrize("change,over,status,needle", ROPE_REFUSALS[1:-6] + [
    ({"v_stride": 8}, {}, B.PA_ERR_INVALID_ARG, "v_stride"),
    ({"head_dim": 64}, {}, B.PA_ERR_INVALID_ARG, "differ"),
    ({"total_tokens": 4}, {}, B.PA_ERR_INVALID_ARG, "differ"),
    ({"num_kv_heads": 1}, {}, B.PA_ERR_INVALID_ARG, "differ"),
    ({"dtype": B.PA_KV_FP16}, {}, B.PA_ERR_INVALID_ARG, "fp16 pools"),
    ({}, {"v": None}, B.PA_ERR_INVALID_ARG, "NULL"),
    ({}, {"kp": _Fake(addr=(1 << 20) + 8)}, B.PA_ERR_INVALID_ARG, "aligned"),
])
def test_norm_rope_append_refusals(change, over, status, needle):
    if "num_q_heads" in change:
        pytest.skip("the two shapes differ first")
    with pytest.raises(B.PaError) as e:
        fused_call(rope(**change), ops.append_shapes(2, 2, 128, 4, 9, 3), **over)
    assert e.value.status == status and needle in str(e.value)


def test_norm_rope_append_needs_scales_and_a_cache_head_dim():
    with pytest.raises(B.PaError, match="4-bit"):
        fused_call(rope(), ops.append_shapes(2, 2, 128, 4, 9, 3, "fp4"))
    with pytest.raises(B.PaError, match="head_dim"):
        fused_call(rope(head_dim=256, q_stride=4096, k_stride=4096, v_stride=4096, q_out_stride=4096),
                   ops.append_shapes(2, 2, 256, 4, 9, 3))


def test_python_shapes():
    qkv = torch.zeros((5, 12 * 64), dtype=torch.bfloat16)
    q, k, v = (x.unflatten(-1, (-1, 64)) for x in qkv.split([8 * 64, 2 * 64, 2 * 64], -1))
    sh = ops.rope_shapes(q, k, v, rope_dim=32, max_position=7, sections=[6, 6, 4])
    assert (sh.q_stride, sh.k_stride, sh.v_stride, sh.q_out_stride, sh.k_out_stride) == (768, 768, 768, 512, 128)
    assert list(sh.sections) == [6, 6, 4] and sh.num_axes == 3
    with pytest.raises(ValueError, match="k"):
        ops.rope_shapes(q, k.transpose(1, 2).contiguous().transpose(1, 2), rope_dim=0)
    with pytest.raises(ValueError, match="v"):
        ops.rope_shapes(q, k, v.float(), rope_dim=0)
    with pytest.raises(ValueError, match="q_out: 5 tokens of stride 512, the shapes are for 5 of 768"):
        ops.qk_norm_rope(ops.rope_shapes(q, k, q_out=q, k_out=k), q, k)
    with pytest.raises(ValueError, match="q_out: 5 tokens of stride 768, the shapes are for 5 of 512"):
        ops.norm_rope_append_kv(ops.rope_shapes(q, k, v), ops.append_shapes(1, 2, 64, 1, 1, 5), q, k, v, *[None] * 5,
                                q_out=q)
    with pytest.raises(ValueError, match="k: 4 tokens"):
        ops.qk_norm_rope(ops.rope_shapes(q, k), q, k[:4])
    t = ops.rope_table(10, 8, theta=100.0, device="cpu")
    assert t.shape == (10, 8) and torch.allclose(t[3, 1], torch.tensor(3 * 100 ** -0.25).cos())


# ----------------------------------------------------------------- tensors that the library would misread

def cache_tensors(kv="fp4", **change):
    """Everything ops.append_kv and ops.gather_kv take for 3 sequences and 10 tokens, 2 heads of 64, 9 pages."""
    t = dict(k_new=torch.zeros((10, 2, 64), dtype=torch.bfloat16), v_new=torch.zeros((10, 2, 64), dtype=torch.bfloat16),
             cu=torch.zeros(4, dtype=torch.int32), start=torch.zeros(3, dtype=torch.int32),
             table=torch.zeros((3, 5), dtype=torch.int32), k_pool=ops.kv_pool(9, 2, 64, kv, "cpu"),
             v_pool=ops.kv_pool(9, 2, 64, kv, "cpu"), k_scale=torch.ones(2), v_scale=torch.ones(2),
             k_out=torch.zeros((10, 2, 64), dtype=torch.bfloat16), v_out=torch.zeros((10, 2, 64), dtype=torch.bfloat16),
             workspace=torch.zeros(256, dtype=torch.uint8))
    t.update(change)
    return t


def ops_cache_call(name, t, kv="fp4"):
    sh = ops.append_shapes(3, 2, 64, 5, 9, 10, kv)
    if name == "append":
        return ops.append_kv(sh, t["k_new"], t["v_new"], t["cu"], t["start"], t["table"], t["k_pool"], t["v_pool"],
                             t["k_scale"], t["v_scale"], t["workspace"], stream=1)
    return ops.gather_kv(sh, t["k_pool"], t["v_pool"], t["cu"], t["start"], t["table"], t["k_scale"], t["v_scale"],
                         t["k_out"], t["v_out"], t["workspace"], stream=1)


PACKED = torch.zeros((10, 6, 64), dtype=torch.bfloat16)
CACHE_TENSORS = [
    ("cu", torch.zeros(4, dtype=torch.int64)), ("cu", torch.zeros(3, dtype=torch.int32)),
    ("start", torch.zeros(3, dtype=torch.int64)), ("start", torch.zeros((3, 2), dtype=torch.int32)[:, 0]),
    ("table", torch.zeros((3, 5), dtype=torch.int64)), ("table", torch.zeros((3, 8), dtype=torch.int32)[:, :5]),
    ("table", torch.zeros((3, 4), dtype=torch.int32)), ("table", torch.zeros((2, 5), dtype=torch.int32)),
    ("table", torch.zeros((5, 3), dtype=torch.int32).T), ("table", torch.zeros(15, dtype=torch.int32)),
    ("k_pool", torch.zeros((8, 2, 2304), dtype=torch.uint8)), ("v_pool", torch.zeros((9, 2, 64, 64), dtype=torch.bfloat16)),
    ("k_pool", torch.zeros((2, 9, 2304), dtype=torch.uint8).transpose(0, 1)),
    ("k_scale", torch.ones(1)), ("v_scale", torch.ones(2, dtype=torch.bfloat16)), ("v_scale", torch.ones(4)[::2]),
    ("workspace", torch.zeros(512, dtype=torch.uint8)[::2]),
]
ROWS = [PACKED[:, 2:4], torch.zeros((9, 2, 64), dtype=torch.bfloat16), torch.zeros((10, 1, 64), dtype=torch.bfloat16),
        torch.zeros((10, 2, 64)), torch.zeros((2, 10, 64), dtype=torch.bfloat16).transpose(0, 1),
        torch.zeros((10, 128), dtype=torch.bfloat16), torch.zeros((10, 2, 64), dtype=torch.float16)]


@pytest.mark.parametrize("name,key,tensor",
                         [(n, k, x) for n in ("append", "gather") for k, x in CACHE_TENSORS]
                         + [("append", k, x) for k in ("k_new", "v_new") for x in ROWS]
                         + [("gather", k, x) for k in ("k_out", "v_out") for x in ROWS])
def test_cache_calls_refuse_tensors_of_another_layout(name, key, tensor):
    with pytest.raises(ValueError, match={"cu": "cu_seqlens", "start": "start_pos", "table": "block_table"}.get(key, key)):
        ops_cache_call(name, cache_tensors(**{key: tensor}))


@pytest.mark.parametrize("name", ["append", "gather"])
@pytest.mark.parametrize("kv,change", [
    ("fp4", {}), ("bf16", {"k_scale": None, "v_scale": None}), ("bf16", {"k_scale": torch.ones(1), "v_scale": None}),
    ("e4m3", {}), ("e4m3", {"k_pool": torch.zeros((9, 2, 64, 64), dtype=torch.uint8)}),
    ("fp4", {"table": torch.zeros((4, 5), dtype=torch.int32)[:, :3]}), ("fp4", {"cu": torch.zeros(9, dtype=torch.int32)}),
    ("fp4", {"k_pool": torch.zeros((12, 2, 2304), dtype=torch.uint8)}),
    ("fp4", {k: torch.zeros((16, 2, 64), dtype=torch.bfloat16) for k in ("k_new", "v_out")}),
])
def test_cache_calls_take_what_the_library_reads_right(name, kv, change):
    """These reach the library: a NULL workspace pointer is what it refuses."""
    t = cache_tensors(kv, **change)
    t["workspace"] = torch.zeros(0, dtype=torch.uint8)
    with pytest.raises(B.PaError):
        ops_cache_call(name, t, kv)


def rope_tensors(tokens=5, **change):
    qkv = torch.zeros((tokens, 12 * 64), dtype=torch.bfloat16)
    q, k, v = (x.unflatten(-1, (-1, 64)) for x in qkv.split([8 * 64, 2 * 64, 2 * 64], -1))
    t = dict(q=q, k=k, v=v, q_weight=torch.ones(64, dtype=torch.bfloat16), k_weight=torch.ones(64, dtype=torch.bfloat16),
             positions=torch.zeros((2, tokens), dtype=torch.int32), cos_sin=torch.zeros((7, 32)),
             q_out=torch.zeros((tokens, 8, 64), dtype=torch.bfloat16), k_out=torch.zeros((tokens, 2, 64), dtype=torch.bfloat16))
    sh = ops.rope_shapes(q, k, v, rope_dim=32, max_position=7, sections=[10, 6])
    t.update(change)
    return sh, t


def ops_rope_call(name, sh, t, workspace=None):
    ws = torch.zeros(0, dtype=torch.uint8) if workspace is None else workspace
    if name == "rope":
        return ops.qk_norm_rope(sh, t["q"], t["k"], t["q_weight"], t["k_weight"], t["positions"], t["cos_sin"], t["q_out"],
                                t["k_out"], ws, stream=1)
    c = cache_tensors()
    ap = ops.append_shapes(3, 2, 64, 5, 9, sh.total_tokens, "fp4")
    return ops.norm_rope_append_kv(sh, ap, t["q"], t["k"], t["v"], c["cu"], t.get("start", c["start"]), c["table"],
                                   t.get("k_pool", c["k_pool"]), c["v_pool"], t["q_weight"], t["k_weight"], t["positions"],
                                   t["cos_sin"], c["k_scale"], c["v_scale"], t["q_out"], ws, stream=1)


ROPE_TENSORS = [
    ("positions", torch.zeros((2, 5), dtype=torch.int64)), ("positions", torch.zeros((1, 5), dtype=torch.int32)),
    ("positions", torch.zeros((5, 2), dtype=torch.int32).T), ("positions", torch.zeros((5, 2), dtype=torch.int32)),
    ("positions", torch.zeros((2, 8), dtype=torch.int32)), ("cos_sin", torch.zeros((7, 32), dtype=torch.bfloat16)),
    ("cos_sin", torch.zeros((7, 32), dtype=torch.float64)), ("cos_sin", torch.zeros((6, 32))),
    ("cos_sin", torch.zeros((14, 16))), ("cos_sin", torch.zeros((32, 7)).T), ("q_weight", torch.ones(64)),
    ("k_weight", torch.ones(64, dtype=torch.float16)), ("q_weight", torch.ones(63, dtype=torch.bfloat16)),
    ("k_weight", torch.ones(128, dtype=torch.bfloat16)[::2]),
    ("q", torch.zeros((5, 12, 64), dtype=torch.float16)[:, :8]), ("q", torch.zeros((5, 12, 64), dtype=torch.bfloat16)[:, :7]),
    ("q", torch.zeros((5, 6, 128), dtype=torch.bfloat16)[:, :4]), ("k", torch.zeros((5, 12, 64), dtype=torch.bfloat16)[:, :1]),
    ("q", torch.zeros((5, 6, 2, 64), dtype=torch.bfloat16).transpose(1, 2).reshape(5, 12, 64)[:, :12:2][:, :8]),
    ("q_out", torch.zeros((5, 4, 64), dtype=torch.bfloat16)), ("q_out", torch.zeros((5, 8, 64), dtype=torch.float16)),
]


@pytest.mark.parametrize("name", ["rope", "fused"])
@pytest.mark.parametrize("key,tensor", ROPE_TENSORS)
def test_rope_calls_refuse_tensors_of_another_layout(name, key, tensor):
    sh, t = rope_tensors(**{key: tensor})
    with pytest.raises(ValueError, match=f"^{key}: "):
        ops_rope_call(name, sh, t)


@pytest.mark.parametrize("name,key,shape", [("rope", "q_out", (1, 4, 64)), ("rope", "k_out", (1, 1, 64)), ("rope", "k", (1, 1, 64)),
                                            ("fused", "v", (1, 1, 64)), ("fused", "q_out", (1, 4, 64)), ("fused", "q", (1, 16, 64))])
def test_one_token_of_other_heads_is_refused(name, key, shape):
    """A single token's stride is never used, so that its heads alone tell a tensor that is too small."""
    sh, t = rope_tensors(1, **{key: torch.zeros(shape, dtype=torch.bfloat16)})
    with pytest.raises(ValueError, match=f"^{key}: "):
        ops_rope_call(name, sh, t)


def test_shapes_of_other_head_counts_are_refused():
    _, t = rope_tensors()
    for key, x in (("v", t["q"]), ("q_out", t["k"]), ("k_out", t["q"])):
        with pytest.raises(ValueError, match=f"^{key}: . heads"):
            ops.rope_shapes(t["q"], t["k"], rope_dim=32, max_position=7, **{key: x})


def test_fused_call_checks_its_cache_and_workspace():
    for key, x in (("start", torch.zeros(3, dtype=torch.int64)), ("k_pool", torch.zeros((8, 2, 2304), dtype=torch.uint8))):
        sh, t = rope_tensors(**{key: x})
        with pytest.raises(ValueError, match="start_pos" if key == "start" else key):
            ops_rope_call("fused", sh, t)
    for name in ("rope", "fused"):
        with pytest.raises(ValueError, match="workspace"):
            ops_rope_call(name, *rope_tensors(), workspace=torch.zeros(512, dtype=torch.uint8)[::2])


@pytest.mark.parametrize("name", ["rope", "fused"])
@pytest.mark.parametrize("change", [{}, {"q_weight": None, "k_weight": None}, {"cos_sin": torch.zeros((9, 32))},
                                    {"positions": torch.zeros((3, 5), dtype=torch.int32)}])
def test_rope_calls_take_what_the_library_reads_right(name, change):
    sh, t = rope_tensors(**change)
    with pytest.raises(B.PaError):
        ops_rope_call(name, sh, t)
    sh.norm = 0  # weights that are not read
    t["q_weight"] = torch.ones(3)
    with pytest.raises(B.PaError):
        ops_rope_call(name, sh, t)
