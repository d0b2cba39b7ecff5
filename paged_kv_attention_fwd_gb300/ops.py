"""Torch-facing helpers around the C ABI.

They allocate outputs, metadata and workspace with torch (device memory only)
and call ``pa_get_metadata`` / ``pa_decode`` / ``pa_prefill``.  All arithmetic
runs in the library's CUDA kernels.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import binding as B


KV_DTYPES = {"bf16": B.PA_KV_BF16, "e4m3": B.PA_KV_FP8_E4M3, "f16": B.PA_KV_FP16, "fp4": B.PA_KV_FP4_E2M1}
_POOL_TORCH = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "f16": torch.float16, "fp4": torch.uint8}


def num_sms(device=None) -> int:
    return torch.cuda.get_device_properties(device or torch.cuda.current_device()).multi_processor_count


def as_bf16(bits: np.ndarray, device) -> torch.Tensor:
    """uint16 bf16 bit patterns -> torch.bfloat16 tensor on `device`."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.to(device).view(torch.bfloat16)


def as_f16(bits: np.ndarray, device) -> torch.Tensor:
    """uint16 fp16 bit patterns -> torch.float16 tensor on `device`."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(torch.float16)


def as_16(bits: np.ndarray, device, dtype: str) -> torch.Tensor:
    return as_f16(bits, device) if dtype == "f16" else as_bf16(bits, device)


def as_e4m3(bits: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits)).to(device).view(torch.float8_e4m3fn)


def _on(stream):
    """What a call allocates is allocated, and cleared, on the stream it runs on."""
    if stream is None:
        return nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        # 0, 1, 2: CUDA's names of the default streams, which wait for one another
        stream = torch.cuda.ExternalStream(handle) if handle > 2 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _output(given, shape, dtype, device, stream):
    if given is not None:
        return given
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


@dataclass
class DecodePlan:
    shapes: B.pa_decode_shapes
    plan: B.pa_decode_plan
    meta: np.ndarray            # host copy
    meta_dev: torch.Tensor      # int32 device copy
    workspace: torch.Tensor     # uint8, zero-filled


def plan_decode(seq_lens_host, block_table_host, num_q_heads: int, num_kv_heads: int, head_dim: int,
                max_pages: int, num_pool_pages: int, kv_dtype: str = "bf16", forced_splits: int = 0,
                ctas_per_sm: int = 0, device="cuda", sms: Optional[int] = None) -> DecodePlan:
    seq_lens_host = np.asarray(seq_lens_host, dtype=np.int32)
    sh = B.pa_decode_shapes(batch=len(seq_lens_host), num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                            head_dim=head_dim, page_size=64, max_pages_per_seq=max_pages,
                            num_pool_pages=num_pool_pages,
                            kv_dtype=KV_DTYPES[kv_dtype],
                            num_sms=sms if sms is not None else num_sms(device), ctas_per_sm=ctas_per_sm,
                            forced_splits=forced_splits)
    meta, plan = B.pa_get_metadata(seq_lens_host, block_table_host, sh)
    meta_dev = torch.from_numpy(meta).to(device)
    ws = torch.zeros(max(plan.workspace_bytes, B.PA_STATUS_BYTES), dtype=torch.uint8, device=device)
    return DecodePlan(sh, plan, meta, meta_dev, ws)


def decode(p: DecodePlan, q, k_pool, v_pool, block_table, seq_lens, scale: float, k_scale=None, v_scale=None,
           out=None, lse=None, stream=None):
    sh = p.shapes
    odt = torch.float16 if sh.kv_dtype == B.PA_KV_FP16 else torch.bfloat16
    out = _output(out, (sh.batch, sh.num_q_heads, sh.head_dim), odt, q.device, stream)
    lse = _output(lse, (sh.batch, sh.num_q_heads), torch.float32, q.device, stream)
    B.pa_decode(sh, p.plan, q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, p.meta_dev, scale, out,
                lse, p.workspace, stream=stream)
    return out, lse


def prefill_shapes(batch, num_q_heads, num_kv_heads, head_dim_qk, head_dim_v, rope_dim, max_seqlen_q, total_q,
                   total_k, max_pages=0, num_pool_pages=0, device="cuda", dtype: str = "bf16") -> B.pa_prefill_shapes:
    return B.pa_prefill_shapes(batch=batch, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                               head_dim_qk=head_dim_qk, head_dim_v=head_dim_v, rope_dim=rope_dim,
                               max_seqlen_q=max_seqlen_q, total_q=total_q, total_k=total_k, page_size=64,
                               max_pages_per_seq=max_pages, num_pool_pages=num_pool_pages,
                               num_sms=num_sms(device), dtype=B.PA_KV_FP16 if dtype == "f16" else B.PA_KV_BF16)


def prefill_mla_fp8(inp, device, causal: bool = True, qo_offset=None, stream=None):
    """pa_prefill_mla_fp8 on an ``MlaE4m3Inputs`` batch (host arrays copied to
    ``device``).  Returns (out bf16, lse fp32, workspace, shapes)."""
    dev = torch.device(device)
    t8 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    sh = B.pa_prefill_shapes(batch=inp.batch, num_q_heads=inp.num_q_heads, num_kv_heads=inp.num_kv_heads,
                             head_dim_qk=192, head_dim_v=128, rope_dim=64, max_seqlen_q=inp.max_seqlen_q,
                             total_q=int(inp.cu_seqlens_q[-1]), total_k=int(inp.cu_seqlens_k[-1]), page_size=64,
                             max_pages_per_seq=0, num_pool_pages=0, num_sms=num_sms(dev),
                             dtype=B.PA_KV_FP8_E4M3)
    out = torch.empty((sh.total_q, sh.num_q_heads, 128), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((sh.total_q, sh.num_q_heads), dtype=torch.float32, device=dev)
    ws = torch.zeros(B.pa_prefill_workspace_size(sh), dtype=torch.uint8, device=dev)
    qo = qo_offset if qo_offset is not None else inp.qo_offset
    B.pa_prefill_mla_fp8(sh, t8(inp.q_nope), as_bf16(inp.q_rope, dev), t8(inp.q_scale), t8(inp.k_nope),
                         t8(inp.k_scale), as_bf16(inp.v, dev), as_bf16(inp.k_rope, dev), t8(inp.cu_seqlens_q),
                         t8(inp.cu_seqlens_k), None if qo is None else t8(np.asarray(qo, np.int32)), causal,
                         inp.scale, out, lse, ws, stream=stream)
    return out, lse, ws, sh


def prefill_mla_rope_fp8(inp, device, causal: bool = True, qo_offset=None, stream=None):
    """pa_prefill_mla_rope_fp8 on an ``MlaRopeE4m3Inputs`` batch (host arrays
    copied to ``device``).  Returns (out bf16, lse fp32, workspace, shapes)."""
    dev = torch.device(device)
    t8 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    sh = B.pa_prefill_shapes(batch=inp.batch, num_q_heads=inp.num_q_heads, num_kv_heads=inp.num_kv_heads,
                             head_dim_qk=192, head_dim_v=128, rope_dim=64, max_seqlen_q=inp.max_seqlen_q,
                             total_q=int(inp.cu_seqlens_q[-1]), total_k=int(inp.cu_seqlens_k[-1]), page_size=64,
                             max_pages_per_seq=0, num_pool_pages=0, num_sms=num_sms(dev), dtype=B.PA_KV_BF16)
    out = torch.empty((sh.total_q, sh.num_q_heads, 128), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((sh.total_q, sh.num_q_heads), dtype=torch.float32, device=dev)
    ws = torch.zeros(B.pa_prefill_mla_rope_fp8_workspace_size(sh), dtype=torch.uint8, device=dev)
    qo = qo_offset if qo_offset is not None else inp.qo_offset
    B.pa_prefill_mla_rope_fp8(sh, as_bf16(inp.q, dev), as_bf16(inp.k_nope, dev), as_bf16(inp.v, dev),
                              t8(inp.k_rope), t8(inp.k_rope_scales), t8(inp.cu_seqlens_q), t8(inp.cu_seqlens_k),
                              None if qo is None else t8(np.asarray(qo, np.int32)), causal, inp.scale, out, lse, ws,
                              stream=stream)
    return out, lse, ws, sh


def prefill(sh: B.pa_prefill_shapes, q, k, v, cu_seqlens_q, cu_seqlens_k, scale: float, causal: bool = True,
            block_table=None, k_rope=None, qo_offset=None, out=None, lse=None, workspace=None, stream=None):
    dev = q.device
    odt = torch.float16 if sh.dtype == B.PA_KV_FP16 else torch.bfloat16
    out = _output(out, (sh.total_q, sh.num_q_heads, sh.head_dim_v), odt, dev, stream)
    lse = _output(lse, (sh.total_q, sh.num_q_heads), torch.float32, dev, stream)
    if workspace is None:
        with _on(stream):
            workspace = torch.zeros(B.pa_prefill_workspace_size(sh), dtype=torch.uint8, device=dev)
    B.pa_prefill(sh, q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, block_table, qo_offset, causal, scale, out, lse,
                 workspace, stream=stream)
    return out, lse, workspace


def kv_pool(num_pages: int, num_kv_heads: int, head_dim: int, kv_dtype: str = "bf16", device="cuda") -> torch.Tensor:
    """A zero-filled K or V pool: [num_pages, Hk, 64, D], or uint8
    [num_pages, Hk, slab bytes] for 4-bit pages."""
    tail = ((B.pa_page_slab_bytes(head_dim, B.PA_KV_FP4_E2M1),) if kv_dtype == "fp4" else (64, head_dim))
    return torch.zeros((num_pages, num_kv_heads, *tail), dtype=_POOL_TORCH[kv_dtype], device=device)


def append_shapes(batch: int, num_kv_heads: int, head_dim: int, max_pages: int, num_pool_pages: int, total_new: int,
                  kv_dtype: str = "bf16") -> B.pa_append_shapes:
    return B.pa_append_shapes(batch=batch, num_kv_heads=num_kv_heads, head_dim=head_dim, page_size=64,
                              max_pages_per_seq=max_pages, num_pool_pages=num_pool_pages, total_new=total_new,
                              kv_dtype=KV_DTYPES[kv_dtype])


# The library sees addresses only: a tensor of another type, shape, layout or
# device than a call takes it to be would be misread, or read or written past
# its end, without an error.  The helpers below refuse such tensors.

def _refuse(name: str, x, expected: str):
    raise ValueError(f"{name}: {x.dtype} {tuple(x.shape)} with strides {tuple(x.stride())} on {x.device}, expected {expected}")


def _check_flat(name: str, x, dtype, count: int, device, what: str):
    """A contiguous tensor of at least `count` elements."""
    if x.dtype != dtype or x.device != device or not x.is_contiguous() or x.numel() < count:
        _refuse(name, x, f"contiguous {what} of {dtype} on {device}")


def _check_rows(name: str, x, sh: B.pa_append_shapes, device):
    """Ragged 16-bit rows [total_new, Hk, D]; a longer buffer will do."""
    dtype = torch.float16 if sh.kv_dtype == B.PA_KV_FP16 else torch.bfloat16
    if x.dim() != 3 or x.shape[0] < sh.total_new or tuple(x.shape[1:]) != (sh.num_kv_heads, sh.head_dim):
        _refuse(name, x, f"[{sh.total_new}, {sh.num_kv_heads}, {sh.head_dim}]")
    _check_flat(name, x, dtype, 0, device, f"[{sh.total_new}, {sh.num_kv_heads}, {sh.head_dim}]")


def _check_cache(sh: B.pa_append_shapes, device, k_pool, v_pool, k_scale, v_scale, cu_seqlens, start_pos, block_table,
                 workspace):
    """What every call on a paged cache takes."""
    slab = B.pa_page_slab_bytes(sh.head_dim, sh.kv_dtype)
    types = {B.PA_KV_BF16: (torch.bfloat16,), B.PA_KV_FP16: (torch.float16,),
             B.PA_KV_FP8_E4M3: (torch.float8_e4m3fn, torch.uint8), B.PA_KV_FP4_E2M1: (torch.uint8,)}.get(sh.kv_dtype, ())
    for name, x in (("k_pool", k_pool), ("v_pool", v_pool)):
        if (x.dtype not in types or x.device != device or not x.is_contiguous()
                or x.numel() * x.element_size() < sh.num_pool_pages * sh.num_kv_heads * slab):
            _refuse(name, x, f"{sh.num_pool_pages} contiguous pages of {sh.num_kv_heads} heads of {slab} bytes, "
                             f"{' or '.join(map(str, types))} on {device}")
    if sh.kv_dtype in (B.PA_KV_FP8_E4M3, B.PA_KV_FP4_E2M1):
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if x is not None:
                _check_flat(name, x, torch.float32, sh.num_kv_heads, device, f"[{sh.num_kv_heads}]")
    _check_flat("cu_seqlens", cu_seqlens, torch.int32, sh.batch + 1, device, f"[{sh.batch + 1}]")
    _check_flat("start_pos", start_pos, torch.int32, sh.batch, device, f"[{sh.batch}]")
    t = block_table
    if (t.dtype != torch.int32 or t.device != device or t.dim() != 2 or t.shape[0] < sh.batch
            or (t.shape[1] > 1 and t.stride(1) != 1) or (sh.batch > 1 and t.stride(0) != sh.max_pages_per_seq)
            or (sh.batch == 1 and t.shape[1] < sh.max_pages_per_seq)):
        _refuse("block_table", t, f"{sh.batch} rows of {sh.max_pages_per_seq} int32, one behind the other, on {device}")
    if workspace is not None:
        _check_flat("workspace", workspace, workspace.dtype, 0, device, "bytes")


def _status(workspace, device, stream):
    if workspace is not None:
        return workspace
    with _on(stream):
        return torch.zeros(B.PA_STATUS_BYTES, dtype=torch.uint8, device=device)


def append_kv(sh: B.pa_append_shapes, k_new, v_new, cu_seqlens_new, start_pos, block_table, k_pool, v_pool,
              k_scale=None, v_scale=None, workspace=None, stream=None):
    """Write new tokens' keys and values, contiguous [total_new, Hk, D], into
    their pages.  Returns the workspace."""
    if sh.batch > 0 and sh.total_new > 0:
        _check_rows("k_new", k_new, sh, k_new.device)
        _check_rows("v_new", v_new, sh, k_new.device)
        _check_cache(sh, k_new.device, k_pool, v_pool, k_scale, v_scale, cu_seqlens_new, start_pos, block_table, workspace)
    workspace = _status(workspace, k_new.device, stream)
    B.pa_append_kv(sh, k_new, v_new, cu_seqlens_new, start_pos, block_table, k_pool, v_pool, k_scale, v_scale,
                   workspace, stream=stream)
    return workspace


def gather_kv(sh: B.pa_append_shapes, k_pool, v_pool, cu_seqlens, start_pos, block_table, k_scale=None, v_scale=None,
              k_out=None, v_out=None, workspace=None, stream=None):
    """Rows of a paged cache as ragged [total_new, Hk, D] tensors (fp16 for
    fp16 pools, else bf16).  Returns (k_out, v_out, workspace)."""
    dt = torch.float16 if sh.kv_dtype == B.PA_KV_FP16 else torch.bfloat16
    shape = (sh.total_new, sh.num_kv_heads, sh.head_dim)
    if sh.batch > 0 and sh.total_new > 0:
        _check_cache(sh, k_pool.device, k_pool, v_pool, k_scale, v_scale, cu_seqlens, start_pos, block_table, workspace)
        for name, x in (("k_out", k_out), ("v_out", v_out)):
            if x is not None:
                _check_rows(name, x, sh, k_pool.device)
    k_out = _output(k_out, shape, dt, k_pool.device, stream)
    v_out = _output(v_out, shape, dt, k_pool.device, stream)
    workspace = _status(workspace, k_pool.device, stream)
    B.pa_gather_kv(sh, k_pool, v_pool, k_scale, v_scale, cu_seqlens, start_pos, block_table, k_out, v_out, workspace,
                   stream=stream)
    return k_out, v_out, workspace


def rope_table(max_position: int, rope_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos_sin for pa_qk_norm_rope: fp32 [max_position, rope_dim], angles
    position * theta^(-2i / rope_dim) taken in fp64."""
    pairs = rope_dim // 2
    freq = theta ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    angle = torch.arange(max_position, dtype=torch.float64)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float().to(device)


def rope_shapes(q, k, v=None, rope_dim: int = 0, max_position: int = 0, interleaved: bool = False, sections=None,
                norm: bool = True, eps: float = 1e-6, q_out=None, k_out=None) -> B.pa_rope_shapes:
    """Shapes of pa_qk_norm_rope for q [T, Hq, D], k and v [T, Hk, D] (slices of
    a packed projection keep their token stride); outputs not given are
    contiguous.  sections: pairs per position axis (default: one axis)."""
    t, hq, d = q.shape
    hk = k.shape[1]
    for name, x in (("q", q), ("k", k), ("v", v), ("q_out", q_out), ("k_out", k_out)):
        if x is not None and (x.shape[0] != t or x.shape[2] != d or (x.shape[1] > 1 and x.stride(1) != d)
                              or x.stride(2) != 1 or x.dtype != q.dtype):
            raise ValueError(f"{name}: heads must be contiguous rows of q's head_dim and type, one per token")
        if x is not None and x.shape[1] != (hq if name in ("q", "q_out") else hk):
            raise ValueError(f"{name}: {x.shape[1]} heads, {hq} query and {hk} key heads given")
    sections = list(sections) if sections is not None else [rope_dim // 2]

    def step(x, heads):  # a single token's stride is never used
        return heads * d if x is None or t <= 1 else x.stride(0)

    sh = B.pa_rope_shapes(total_tokens=t, num_q_heads=hq, num_kv_heads=hk, head_dim=d, rope_dim=rope_dim,
                          interleaved=int(interleaved), num_axes=len(sections), max_position=max_position,
                          dtype={torch.bfloat16: B.PA_KV_BF16, torch.float16: B.PA_KV_FP16}[q.dtype], norm=int(norm),
                          eps=eps, q_stride=step(q, hq), k_stride=step(k, hk), v_stride=step(v, hk),
                          q_out_stride=step(q_out, hq), k_out_stride=step(k_out, hk))
    for i, n in enumerate(sections[:3]):
        sh.sections[i] = n
    return sh


def _check_steps(sh: B.pa_rope_shapes, **tensors):
    """Tensors as the shapes describe them: a step other than theirs would reach past an output."""
    dtype = torch.float16 if sh.dtype == B.PA_KV_FP16 else torch.bfloat16
    for name, x in tensors.items():
        step, d = getattr(sh, name + "_stride"), sh.head_dim
        if x.shape[0] != sh.total_tokens or (sh.total_tokens > 1 and x.shape[1] > 0 and x.stride(0) != step):
            raise ValueError(f"{name}: {x.shape[0]} tokens of stride {x.stride(0)}, the shapes are for "
                             f"{sh.total_tokens} of {step}")
        heads = sh.num_q_heads if name in ("q", "q_out") else sh.num_kv_heads
        if (tuple(x.shape[1:]) != (heads, d) or x.dtype != dtype or x.device != tensors["q"].device
                or (heads > 1 and x.stride(1) != d) or (heads > 0 and x.stride(2) != 1)):
            _refuse(name, x, f"{heads} contiguous heads of {d} of {dtype} on {tensors['q'].device}")


def _check_rope(sh: B.pa_rope_shapes, q, q_weight, k_weight, positions, cos_sin):
    if sh.norm:
        for name, x in (("q_weight", q_weight), ("k_weight", k_weight)):
            if x is not None:
                _check_flat(name, x, q.dtype, sh.head_dim, q.device, f"[{sh.head_dim}]")
    if sh.rope_dim == 0:  # neither is read
        return
    if positions is not None:
        _check_flat("positions", positions, torch.int32, sh.num_axes * sh.total_tokens, q.device,
                    f"[{sh.num_axes}, {sh.total_tokens}]")
        if positions.shape[-1] != sh.total_tokens:
            _refuse("positions", positions, f"[{sh.num_axes}, {sh.total_tokens}]")
    if cos_sin is not None:
        _check_flat("cos_sin", cos_sin, torch.float32, sh.max_position * sh.rope_dim, q.device,
                    f"[{sh.max_position}, {sh.rope_dim}]")
        if cos_sin.shape[-1] != sh.rope_dim:
            _refuse("cos_sin", cos_sin, f"[{sh.max_position}, {sh.rope_dim}]")


def qk_norm_rope(sh: B.pa_rope_shapes, q, k, q_weight=None, k_weight=None, positions=None, cos_sin=None, q_out=None,
                 k_out=None, workspace=None, stream=None):
    """RMS norm of every head, then the rotation.  Returns (q_out, k_out, workspace)."""
    q_out = _output(q_out, q.shape, q.dtype, q.device, stream)
    k_out = _output(k_out, k.shape, k.dtype, k.device, stream)
    _check_steps(sh, q=q, k=k, q_out=q_out, k_out=k_out)
    _check_rope(sh, q, q_weight, k_weight, positions, cos_sin)
    if workspace is not None:
        _check_flat("workspace", workspace, workspace.dtype, 0, q.device, "bytes")
    workspace = _status(workspace, q.device, stream)
    B.pa_qk_norm_rope(sh, q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, workspace, stream=stream)
    return q_out, k_out, workspace


def norm_rope_append_kv(sh: B.pa_rope_shapes, append: B.pa_append_shapes, q, k, v, cu_seqlens_new, start_pos,
                        block_table, k_pool, v_pool, q_weight=None, k_weight=None, positions=None, cos_sin=None,
                        k_scale=None, v_scale=None, q_out=None, workspace=None, stream=None):
    """qk_norm_rope with the keys and values going straight into their pages.
    Returns (q_out, workspace)."""
    q_out = _output(q_out, q.shape, q.dtype, q.device, stream)
    _check_steps(sh, q=q, k=k, v=v, q_out=q_out)
    _check_rope(sh, q, q_weight, k_weight, positions, cos_sin)
    if append.batch > 0 and sh.total_tokens > 0:
        _check_cache(append, q.device, k_pool, v_pool, k_scale, v_scale, cu_seqlens_new, start_pos, block_table, workspace)
    workspace = _status(workspace, q.device, stream)
    B.pa_norm_rope_append_kv(sh, append, q, k, v, q_weight, k_weight, positions, cos_sin, cu_seqlens_new, start_pos,
                             block_table, q_out, k_pool, v_pool, k_scale, v_scale, workspace, stream=stream)
    return q_out, workspace
