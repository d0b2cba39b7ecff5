"""Host-side checks of the calls around a latent cache: bad arguments are
refused with the documented status, and tensors that the library would misread
with a ValueError, before anything is enqueued (no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops
from paged_kv_attention_fwd_gb300.build import build

from .test_abi import _Fake

NULL, ODD = None, _Fake(addr=(1 << 20) + 8)


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def project(**over):
    return B.pa_mla_project_shapes(**{**dict(total_tokens=4, num_heads=2, head_dim=128, latent_dim=512, rope_dim=64, dtype=0,
                                             max_position=100, in_stride=2 * 512, out_stride=2 * 576,
                                             w_stride=256 * 512), **over})


def cache(**over):
    return B.pa_mla_cache_shapes(**{**dict(batch=2, latent_dim=512, rope_dim=64, page_size=64, max_pages_per_seq=3,
                                           num_pool_pages=9, total_new=5, dtype=0, norm=1, max_position=100, eps=1e-6,
                                           kv_stride=576), **over})


def attend(**over):
    return B.pa_mla_decode_shapes(**{**dict(batch=2, num_q_heads=16, q_len=1, latent_dim=512, rope_dim=64, page_size=64,
                                            max_pages_per_seq=3, num_pool_pages=9, num_sms=152, dtype=0), **over})


CALLS = {
    "query": ("pa_mla_query", project, ["q", "w", "positions", "cos_sin", "out"]),
    "output": ("pa_mla_output", project, ["o", "w", "out"]),
    "append": ("pa_mla_append_kv", cache, ["kv", "weight", "positions", "cos_sin", "cu", "start", "table", "pool"]),
    "gather": ("pa_mla_gather_kv", cache, ["pool", "cu", "start", "table", "latent", "rope"]),
    "decode": ("pa_mla_decode", attend, ["q", "pool", "table", "lens", "scale", "out", "lse"]),
}


def call(name, shapes, over=None, size=1 << 30):
    function, _, names = CALLS[name]
    args = {n: _Fake() for n in names + ["workspace"]}
    if "scale" in args:
        args["scale"] = 0.1
    args.update(over or {})
    getattr(B, function)(shapes, *[args[n] for n in names], args["workspace"], size, stream=0)


ROW = [({"latent_dim": 256}, B.PA_ERR_UNSUPPORTED, "latent_dim"), ({"rope_dim": 32}, B.PA_ERR_UNSUPPORTED, "rope_dim"),
       ({"dtype": B.PA_KV_FP8_E4M3}, B.PA_ERR_UNSUPPORTED, "bf16 or fp16"),
       ({"dtype": B.PA_KV_FP4_E2M1}, B.PA_ERR_UNSUPPORTED, "bf16 or fp16"), ({"dtype": 9}, B.PA_ERR_INVALID_ARG, "dtype")]
PAGES = [({"page_size": 32}, B.PA_ERR_INVALID_ARG, "page_size"), ({"max_pages_per_seq": 0}, B.PA_ERR_INVALID_ARG, "max_pages"),
         ({"num_pool_pages": 0}, B.PA_ERR_INVALID_ARG, "num_pool_pages")]
SHAPES = {
    "query": ROW + [({"head_dim": 64}, B.PA_ERR_UNSUPPORTED, "head_dim"), ({"num_heads": 0}, B.PA_ERR_INVALID_ARG, "num_heads"),
                    ({"total_tokens": -1}, B.PA_ERR_INVALID_ARG, "total_tokens"),
                    ({"in_stride": 376}, B.PA_ERR_INVALID_ARG, "in_stride"), ({"in_stride": 388}, B.PA_ERR_INVALID_ARG, "in_stride"),
                    ({"out_stride": 1148}, B.PA_ERR_INVALID_ARG, "out_stride"),
                    ({"w_stride": 128 * 512 - 8}, B.PA_ERR_INVALID_ARG, "w_stride"),
                    ({"max_position": 0}, B.PA_ERR_INVALID_ARG, "max_position"),
                    ({"total_tokens": 2 ** 31 - 1}, B.PA_ERR_UNSUPPORTED, "total_tokens")],
    "output": ROW + [({"in_stride": 1016}, B.PA_ERR_INVALID_ARG, "in_stride"), ({"out_stride": 250}, B.PA_ERR_INVALID_ARG, "out_stride")],
    "append": ROW + PAGES + [({"batch": -1}, B.PA_ERR_INVALID_ARG, "batch"), ({"total_new": -1}, B.PA_ERR_INVALID_ARG, "total_new"),
                             ({"norm": 2}, B.PA_ERR_INVALID_ARG, "norm"), ({"eps": -1.0}, B.PA_ERR_INVALID_ARG, "eps"),
                             ({"eps": float("nan")}, B.PA_ERR_INVALID_ARG, "eps"),
                             ({"kv_stride": 568}, B.PA_ERR_INVALID_ARG, "kv_stride"), ({"kv_stride": 580}, B.PA_ERR_INVALID_ARG, "kv_stride"),
                             ({"max_position": 0}, B.PA_ERR_INVALID_ARG, "max_position"),
                             ({"total_new": 2 ** 31 - 1}, B.PA_ERR_UNSUPPORTED, "total_new")],
    "gather": ROW + PAGES + [({"total_new": -2}, B.PA_ERR_INVALID_ARG, "total_new")],
    "decode": ROW + PAGES + [({"batch": -1}, B.PA_ERR_INVALID_ARG, "batch"), ({"num_q_heads": 0}, B.PA_ERR_INVALID_ARG, "num_q_heads"),
                             ({"q_len": 0}, B.PA_ERR_INVALID_ARG, "q_len"), ({"num_sms": 0}, B.PA_ERR_INVALID_ARG, "num_sms"),
                             ({"num_q_heads": 40000, "q_len": 2}, B.PA_ERR_UNSUPPORTED, "65536"),
                             ({"batch": 2 ** 30}, B.PA_ERR_UNSUPPORTED, "2^31"),
                             ({"batch": 2 ** 20, "max_pages_per_seq": 2 ** 12}, B.PA_ERR_UNSUPPORTED, "max_pages_per_seq"),
                             ({"num_pool_pages": 2 ** 25}, B.PA_ERR_UNSUPPORTED, "pool rows")],
}
OPTIONAL = {"query": ["cos_sin"], "output": [], "append": ["weight", "positions", "cos_sin"], "gather": [], "decode": ["lse"]}
ALIGNED = {"query": ["q", "w", "out", "cos_sin", "workspace"], "output": ["o", "w", "out", "workspace"],
           "append": ["kv", "weight", "cos_sin", "pool", "workspace"], "gather": ["pool", "latent", "rope", "workspace"],
           "decode": ["q", "pool", "out", "workspace"]}


@pytest.mark.parametrize("name,over,status,needle", [(n, *c) for n, cases in SHAPES.items() for c in cases])
def test_shapes_are_refused(name, over, status, needle):
    with pytest.raises(B.PaError) as e:
        call(name, CALLS[name][1](**over))
    assert e.value.status == status and needle in str(e.value)


@pytest.mark.parametrize("name", CALLS)
def test_null_and_unaligned_pointers_are_refused(name):
    shapes = CALLS[name][1]()
    for n in CALLS[name][2] + ["workspace"]:
        if n != "scale" and n not in OPTIONAL[name]:
            with pytest.raises(B.PaError, match="NULL"):
                call(name, shapes, {n: NULL})
    for n in ALIGNED[name]:
        with pytest.raises(B.PaError, match="16-byte"):
            call(name, shapes, {n: ODD})
    with pytest.raises(B.PaError) as e:
        call(name, shapes, size=255)
    assert e.value.status == B.PA_ERR_WORKSPACE
    with pytest.raises(B.PaError, match="shapes"):
        B._check(getattr(B.lib(), CALLS[name][0])(None, *[0.0 if n == "scale" else None for n in CALLS[name][2]], None, 0, None))


def test_scale_and_workspace_of_decode():
    for scale in (float("inf"), float("nan")):
        with pytest.raises(B.PaError, match="scale"):
            call("decode", attend(), {"scale": scale})
    need = B.pa_mla_decode_workspace_size(attend())
    assert need >= 2 * 152 * 64 * 512 * 4 and need == B.pa_mla_decode_workspace_size(attend(batch=500, num_q_heads=128, q_len=4))
    assert B.pa_mla_decode_workspace_size(attend(num_sms=10)) < need
    with pytest.raises(B.PaError) as e:
        call("decode", attend(), size=need - 1)
    assert e.value.status == B.PA_ERR_WORKSPACE
    assert B.lib().pa_mla_decode_workspace_size(None) == B.PA_STATUS_BYTES
    assert B.lib().pa_mla_decode_workspace_size(ctypes.byref(attend(num_sms=-1))) == B.PA_STATUS_BYTES


@pytest.mark.parametrize("name,over", [("query", {"total_tokens": 0}), ("output", {"total_tokens": 0}), ("append", {"batch": 0}),
                                       ("append", {"total_new": 0}), ("gather", {"total_new": 0}), ("decode", {"batch": 0})])
def test_empty_calls_do_nothing(name, over):
    nothing = {n: NULL for n in CALLS[name][2] + ["workspace"] if n != "scale"}
    call(name, CALLS[name][1](**over), nothing, 0)


# ----------------------------------------------------------------- tensors that would be misread

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return t(*shape, dtype=torch.int32)


GOOD = {
    "query": dict(q=t(4, 2, 192), w_uk=t(2, 256, 512)[:, :128], positions=i32(4), cos_sin=t(100, 64, dtype=torch.float32),
                  q_out=t(4, 2, 576), workspace=t(256, dtype=torch.uint8)),
    "output": dict(o=t(4, 2, 512), w_uv=t(2, 256, 512)[:, 128:], out=t(4, 2, 128), workspace=t(256, dtype=torch.uint8)),
    "append": dict(sh=cache(kv_stride=640), kv_new=t(5, 640)[:, 64:], cu_seqlens_new=i32(3), start_pos=i32(2), block_table=i32(2, 3),
                   pool=t(9, 64, 576), weight=t(512), positions=i32(5), cos_sin=t(100, 64, dtype=torch.float32),
                   workspace=t(256, dtype=torch.uint8)),
    "gather": dict(sh=cache(), pool=t(9, 64, 576), cu_seqlens=i32(3), start_pos=i32(2), block_table=i32(2, 3),
                   latent_out=t(5, 512), rope_out=t(5, 1, 64), workspace=t(256, dtype=torch.uint8)),
    "decode": dict(sh=attend(), q=t(2, 16, 576), pool=t(9, 64, 576), block_table=i32(2, 3), seq_lens=i32(2), scale=0.1,
                   out=t(2, 16, 512), lse=t(2, 16, dtype=torch.float32), workspace=t(256, dtype=torch.uint8)),
}
FUNCTIONS = {"query": ops.mla_query, "output": ops.mla_output, "append": ops.mla_append_kv, "gather": ops.mla_gather_kv,
             "decode": ops.mla_decode}
BAD = [
    ("query", "q", t(4, 2, 128)), ("query", "q", t(4, 2, 192, dtype=torch.float32)), ("query", "q", t(4, 2, 384)[..., ::2]),
    ("query", "q", t(4, 384)), ("query", "q", t(2, 4, 192).transpose(0, 1)),
    ("query", "w_uk", t(2, 512, 128)), ("query", "w_uk", t(3, 128, 512)), ("query", "w_uk", t(2, 512, 128).transpose(1, 2)),
    ("query", "w_uk", t(2, 128, 512, dtype=torch.float16)), ("query", "positions", i32(3)),
    ("query", "positions", t(4, dtype=torch.int64)), ("query", "cos_sin", t(100, 32, dtype=torch.float32)),
    ("query", "cos_sin", t(100, 64)), ("query", "q_out", t(4, 2, 512)), ("query", "q_out", t(4, 2, 576, dtype=torch.float16)),
    ("output", "o", t(4, 2, 576)), ("output", "w_uv", t(2, 128, 1024)[..., ::2]), ("output", "out", t(4, 2, 64)),
    ("output", "out", t(4, 2, 128, dtype=torch.float16)), ("output", "workspace", t(512, dtype=torch.uint8)[::2]),
    ("append", "kv_new", t(4, 640)[:, 64:]), ("append", "kv_new", t(5, 576)), ("append", "kv_new", t(5, 640, dtype=torch.float16)[:, 64:]),
    ("append", "kv_new", t(576, 640)[:, :5].T), ("append", "cu_seqlens_new", i32(2)), ("append", "start_pos", t(2, dtype=torch.int64)),
    ("append", "block_table", i32(2, 4)), ("append", "block_table", i32(1, 3)), ("append", "pool", t(8, 64, 576)),
    ("append", "pool", t(9, 64, 576, dtype=torch.float16)), ("append", "weight", t(256)), ("append", "weight", t(512, dtype=torch.float32)),
    ("append", "positions", i32(4)), ("append", "cos_sin", t(99, 64, dtype=torch.float32)),
    ("gather", "pool", t(9, 576, 64).transpose(1, 2)), ("gather", "latent_out", t(4, 512)), ("gather", "rope_out", t(5, 128)[:, ::2]),
    ("gather", "latent_out", t(5, 512, dtype=torch.float32)), ("gather", "cu_seqlens", i32(6)[::2]),
    ("decode", "q", t(2, 8, 576)), ("decode", "q", t(2, 16, 640)[..., :576]), ("decode", "q", t(2, 16, 576, dtype=torch.float16)),
    ("decode", "pool", t(9, 64, 512)), ("decode", "seq_lens", t(2, dtype=torch.int64)), ("decode", "seq_lens", i32(1)),
    ("decode", "out", t(2, 16, 256)), ("decode", "lse", t(2, 16)), ("decode", "block_table", i32(2, 5)[:, :3]),
]


@pytest.mark.parametrize("name,key,tensor", BAD)
def test_tensors_of_another_layout_are_refused(name, key, tensor):
    with pytest.raises(ValueError, match="input|weights|output|" + key.replace("_new", "")):
        FUNCTIONS[name](**{**GOOD[name], key: tensor})


@pytest.mark.parametrize("name", CALLS)
def test_tensors_as_the_library_reads_them_reach_it(name, monkeypatch):
    seen = []
    monkeypatch.setattr(B, CALLS[name][0], lambda *a, **k: seen.append(a))
    FUNCTIONS[name](**GOOD[name])
    assert len(seen) == 1


def test_strides_of_slices():
    packed = t(4, 2 * 192 + 64)
    sh = ops.mla_query_shapes(packed[:, :384].unflatten(-1, (2, 192)), t(2, 256, 512)[:, :128], 7, True)
    assert (sh.in_stride, sh.out_stride, sh.w_stride, sh.max_position, sh.interleaved) == (448, 1152, 256 * 512, 7, 1)
    sh = ops.mla_output_shapes(t(1, 2, 512), t(2, 128, 512), t(4, 2, 128)[:1])
    assert (sh.in_stride, sh.out_stride, sh.w_stride, sh.total_tokens) == (1024, 256, 128 * 512, 1)
