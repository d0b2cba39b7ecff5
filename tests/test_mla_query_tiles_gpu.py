"""pa_mla_query where an SM keeps a head's weights for several tiles of tokens:
tiles with padding among their tokens, tiles of nothing else, and last tiles of
a few tokens, between tiles that leave whole."""
import pytest
import torch

from paged_kv_attention_fwd_gb300 import binding as B
from paged_kv_attention_fwd_gb300 import ops

from .test_mla_gpu import DEV, HALF, T16, TINY, gpu, near, normal, ok, product_tol, turned  # noqa: F401

pytestmark = pytest.mark.gpu
HEADS = 160  # two tiles of them are more than two an SM


@pytest.mark.parametrize("t", [129, 143, 144, 260, 400, 641])
@pytest.mark.parametrize("padded", ["none", "some", "a tile", "all but one", "out of range"])
@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("f16", True)])
def test_padding_and_short_last_tiles(t, padded, dtype, inter):
    q, w = normal((t, HEADS, 192), 1, dtype), normal((HEADS, 128, 512), 2, dtype) * 0.05
    angles = ops.rope_table(500, 64)
    at = (torch.arange(t, device=DEV, dtype=torch.int32) * 7) % 500
    if padded == "some":
        at[[0, 5, 127, t - 1]] = -1
    elif padded == "a tile":
        at[128:256] = -7
    elif padded == "all but one":
        at[torch.arange(t, device=DEV) != t - 2] = -1
    elif padded == "out of range":
        at[[3, 128]] = 500
    live = (at >= 0) & (at < 500)
    q[~live] = float("nan")
    out = torch.full((t + 1, HEADS, 576), 7.0, dtype=T16[dtype], device=DEV)
    _, ws = ops.mla_query(q, w, at, angles, inter, q_out=out[:t])
    assert B.pa_check_status(ws) == (B.PA_ERR_DEVICE_BOUNDS if padded == "out of range" else B.PA_OK)
    assert (out[:t][~live] == 7).all() and (out[t] == 7).all()
    x = q[live]
    want = torch.einsum("thi,hik->thk", x[..., :128].double(), w.double())
    reach = torch.einsum("thi,hik->thk", x[..., :128].double().abs(), w.double().abs())
    got = out[:t][live]
    near(got[..., :512], want, product_tol(want, reach, 128, dtype))
    want = turned(x[..., 128:], at[live], angles, inter)
    near(got[..., 512:], want, HALF[dtype] * want.abs() + 2.0 ** -22 * x[..., 128:].double().abs().amax() + TINY[dtype])
