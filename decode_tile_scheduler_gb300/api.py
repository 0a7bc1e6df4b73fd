"""PyTorch-facing helpers: build the C-ABI parameter structs from tensors,
allocate outputs and workspaces with torch, and launch on the tensors' device, on
torch's current CUDA stream there.  Memory and streams only -- the computation is libfia's.
"""
from __future__ import annotations

import contextlib
import math
from typing import Optional

import torch

from . import _abi
from ._abi import FiaParams, SparseParams


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libfia takes CUDA tensors")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (2 us of a call that
# takes 6), and the current device without a look at whether CUDA is up (0.3 us: the
# tensors of a call are on it), where this PyTorch has the accessors.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current_stream(device_index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device_index)
    return torch.cuda.current_stream(device_index).cuda_stream


def _handle(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_HERE = contextlib.nullcontext()


def _on(device: torch.device):
    """Context in which `device` is the current one."""
    return _HERE if device.index == _current_device() else torch.cuda.device(device)


def _launch(device: torch.device, stream, call, *args):
    """call(*args, stream's handle) with `device` as the current one.  libfia launches on
    the current device and asks it for its SMs, whatever device the pointers belong
    to, and the default stream's handle names no device; so every call enters its
    tensors'.  A torch stream of another device is refused (other handles cannot be
    told)."""
    index = device.index
    if stream is None:
        if index == _current_device():
            return call(*args, _current_stream(index))
    else:
        of = getattr(stream, "device", None)
        if isinstance(of, torch.device) and of != device:
            raise ValueError(f"the stream is on {of}, the tensors on {device}")
    with _on(device):
        return call(*args, _current_stream(index) if stream is None else _handle(stream))


def _made_on(stream, device: torch.device):
    """Context in which torch allocates and fills on `stream` (None: the current
    one).  A call that makes its own outputs and workspace and returns enters it:
    made on the current stream, a fill could run behind the call's kernels, and
    the workspace could go to the current stream's next tensor while they run."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _handle(stream)
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def _contig(t: Optional[torch.Tensor], name: str):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def make_fia_params(*, q: torch.Tensor, out: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, num_q_heads: int, num_kv_heads: int, head_dim: int,
                    batch: int, layout: int, max_seqlen_q: int, total_q: int = 0,
                    lse: Optional[torch.Tensor] = None, kv_dtype: int = _abi.KV_BF16,
                    k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None,
                    block_table: Optional[torch.Tensor] = None, block_size: int = 0,
                    num_blocks: int = 0, max_seqlen_kv: int = 0,
                    cu_seqlens_q: Optional[torch.Tensor] = None,
                    seqused_kv: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    mask_mode: int = _abi.MASK_NONE, pre_tokens: int = 0, next_tokens: int = 0,
                    sinks: Optional[torch.Tensor] = None, num_sms: int = 0,
                    kv_layout: int = _abi.KV_LAYOUT_BNBSH,
                    atten_mask: Optional[torch.Tensor] = None,
                    first_tokens: int = 0) -> FiaParams:
    """`kv_dtype` KV_MXFP4: caches of bytes, two E2M1 codes each ([.., D/2]), and scales
    of bytes [pages or B, KV heads, rows, D/32].  `atten_mask`: int8/uint8/bool [B or 1, rows, cols] (nonzero = masked
    out), rows >= the query length, cols a multiple of 16 >= the KV capacity;
    a first dimension of 1 is shared by every batch.  `first_tokens` (band
    mask): keys below it stay visible beside the window."""
    for name, t in (("q", q), ("out", out), ("k_cache", k_cache), ("v_cache", v_cache)):
        _contig(t, name)
    for name, t in (("out", out), ("k_cache", k_cache), ("v_cache", v_cache), ("lse", lse),
                    ("k_scale", k_scale), ("v_scale", v_scale), ("block_table", block_table),
                    ("cu_seqlens_q", cu_seqlens_q), ("seqused_kv", seqused_kv), ("sinks", sinks),
                    ("atten_mask", atten_mask)):
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    if kv_dtype == _abi.KV_MXFP4:  # (bytes: sizes and type are all that tells them from others)
        n, rows = int(k_cache.shape[0]), block_size if block_table is not None else max_seqlen_kv
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype != torch.uint8 or t.numel() != n * rows * num_kv_heads * (head_dim // 2):
                raise ValueError(f"{name}: an MXFP4 cache holds D/2 bytes a row (uint8)")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None or t.dtype not in (torch.uint8, torch.float8_e8m0fnu):
                raise ValueError(f"{name}: an MXFP4 cache has E8M0 scales (uint8, float8_e8m0fnu)")
            _checked(t, name, t.dtype, (n, num_kv_heads, rows, head_dim // 32), k_cache.device)
    p = FiaParams()
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim = batch, num_q_heads, num_kv_heads, head_dim
    p.layout, p.max_seqlen_q, p.total_q = layout, max_seqlen_q, total_q
    p.q, p.out, p.lse = _ptr(q), _ptr(out), _ptr(lse)
    p.k_cache, p.v_cache = _ptr(k_cache), _ptr(v_cache)
    p.k_scale, p.v_scale = _ptr(k_scale), _ptr(v_scale)
    p.kv_dtype = kv_dtype
    p.quant_tile = {_abi.KV_FP8_E4M3: 64, _abi.KV_MXFP4: 32}.get(kv_dtype, 0)
    p.block_table = _ptr(block_table)
    p.max_blocks_per_seq = 0 if block_table is None else int(block_table.shape[1])
    p.block_size, p.num_blocks, p.max_seqlen_kv = block_size, num_blocks, max_seqlen_kv
    p.cu_seqlens_q, p.seqused_kv = _ptr(cu_seqlens_q), _ptr(seqused_kv)
    p.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
    p.mask_mode, p.pre_tokens, p.next_tokens = mask_mode, pre_tokens, next_tokens
    p.sinks = _ptr(sinks)
    p.num_sms = num_sms
    p.kv_layout = kv_layout
    p.first_tokens = _int32(first_tokens, "first_tokens")
    if atten_mask is not None:
        _contig(atten_mask, "atten_mask")
        if atten_mask.dim() != 3 or atten_mask.element_size() != 1:
            raise ValueError("atten_mask must be a 3-d tensor of 1-byte elements")
        p.atten_mask = _ptr(atten_mask)
        p.mask_row_stride = int(atten_mask.stride(1))
        p.mask_batch_stride = 0 if atten_mask.shape[0] == 1 else int(atten_mask.stride(0))
    return p


def params_from_problem(prob, out: torch.Tensor, lse: Optional[torch.Tensor],
                        num_sms: int = 0) -> FiaParams:
    """Parameters for a problem object with the generator's field names
    (B, QN, KVN, D, layout, S_q, T, q, k_cache, ...)."""
    return make_fia_params(
        q=prob.q, out=out, k_cache=prob.k_cache, v_cache=prob.v_cache, num_q_heads=prob.QN,
        num_kv_heads=prob.KVN, head_dim=prob.D, batch=prob.B, layout=prob.layout,
        max_seqlen_q=prob.S_q, total_q=prob.T, lse=lse, kv_dtype=prob.kv_dtype,
        k_scale=prob.k_scale, v_scale=prob.v_scale, block_table=prob.block_table,
        block_size=prob.block_size, num_blocks=prob.num_blocks,
        max_seqlen_kv=0 if prob.block_table is not None else prob.S_kv,
        cu_seqlens_q=prob.cu_seqlens_q, seqused_kv=prob.seqused_kv, scale=prob.scale,
        mask_mode=prob.mask_mode, pre_tokens=prob.pre_tokens, next_tokens=prob.next_tokens,
        sinks=prob.sinks, num_sms=num_sms, kv_layout=getattr(prob, "kv_layout", 0),
        atten_mask=getattr(prob, "atten_mask", None),
        first_tokens=getattr(prob, "first_tokens", 0))


def lse_shape(prob):
    return (prob.T, prob.QN, 1) if prob.layout == _abi.LAYOUT_TND else (prob.B, prob.QN, prob.S_q, 1)


def _outputs(prob, out: Optional[torch.Tensor], lse: Optional[torch.Tensor], with_lse: bool):
    """out and lse of a call: new tensors, or the given ones, whose sizes and types
    the kernels rely on."""
    shape = lse_shape(prob)
    if out is None:
        out = torch.empty_like(prob.q)
    elif out.numel() != prob.q.numel() or out.dtype != prob.q.dtype:
        raise ValueError(f"out must hold q's {tuple(prob.q.shape)} in {prob.q.dtype}")
    if lse is None:
        lse = torch.empty(shape, dtype=torch.float32, device=prob.q.device) if with_lse else None
    elif lse.numel() != math.prod(shape) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of {shape}")
    return out, lse


class FiaCall:
    """One configured FIA call: owns its outputs and workspace (torch
    allocations, made on the stream that is current where the call is) and
    launches plan/execute/run on a stream.  Keep the object until that stream
    has run what was launched: its workspace goes with it."""

    def __init__(self, prob, with_lse: bool = True, num_sms: int = 0, out=None, lse=None):
        dev = self.device = prob.q.device
        self.prob = prob
        self.out, self.lse = _outputs(prob, out, lse, with_lse)
        self.params = params_from_problem(prob, self.out, self.lse, num_sms)
        with _on(dev):
            self.ws_bytes = _abi.fia_get_workspace_size(self.params)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def plan(self, stream=None):
        _launch(self.device, stream, _abi.fia_plan, self.params, self.ws.data_ptr(), self.ws_bytes)

    def execute(self, stream=None):
        _launch(self.device, stream, _abi.fia_execute, self.params, self.ws.data_ptr(),
                self.ws_bytes)

    def run(self, stream=None):
        _launch(self.device, stream, _abi.fia_run, self.params, self.ws.data_ptr(), self.ws_bytes)
        return self.out, self.lse

    def plan_layout(self):
        with _on(self.device):
            return _abi.fia_get_plan_layout(self.params)

    def error_word(self) -> int:
        return int(self.ws[:4].view(torch.int32).item())


def fused_infer_attention(prob, with_lse: bool = True, num_sms: int = 0, stream=None):
    """Run FIA on a problem object; returns (out, lse), made on `stream`."""
    with _made_on(stream, prob.q.device):
        return FiaCall(prob, with_lse=with_lse, num_sms=num_sms).run(stream)


# ----------------------------------------------------------------------------
# a bounded cache: append, attention with key weights, eviction
# ----------------------------------------------------------------------------

def _checked(t: Optional[torch.Tensor], name: str, dtype, shape, device):
    """Device address of a contiguous tensor of that dtype, shape and device."""
    if t is None:
        return None
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    return _ptr(t)


def _state(t: Optional[torch.Tensor], name: str, dtype, batch: int, heads: int, capacity: int,
           device):
    """Address and row stride of a per-key state tensor [batch, heads, n], n >=
    the cache's capacity, rows evenly spaced."""
    if t is None:
        return None, 0
    if t.dtype != dtype or t.dim() != 3 or tuple(t.shape[:2]) != (batch, heads) \
            or t.shape[2] < capacity:
        raise ValueError(f"{name} must be a {dtype} tensor [{batch}, {heads}, >= {capacity}]")
    row = int(t.stride(1)) if heads > 1 else int(t.stride(0))
    if batch == 1 and heads == 1:
        row = max(capacity, 1)  # (one row: any stride)
    if (t.shape[2] > 1 and t.stride(2) != 1) or (batch > 1 and t.stride(0) != heads * row):
        raise ValueError(f"{name}: rows of unit stride, evenly spaced")
    if row < capacity:
        raise ValueError(f"{name}: its rows overlap")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    return _ptr(t), row


def _new_state(like: Optional[torch.Tensor], dtype, batch: int, heads: int, capacity: int, device):
    """A state tensor of zeros with the row stride (and shape) of `like`."""
    if like is None or like.dim() != 3:
        return torch.zeros((batch, heads, capacity), dtype=dtype, device=device)
    row = int(like.stride(1)) if heads > 1 else int(like.stride(0)) if batch > 1 else 0
    row = max(row, int(like.shape[2]))
    return torch.zeros((batch, heads, row), dtype=dtype, device=device)[:, :, :like.shape[2]]


def _int32(x: int, name: str) -> int:
    """An int32 field's value (ctypes would drop the upper bits of a larger one)."""
    if not -(1 << 31) <= int(x) < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits")
    return int(x)


def _one_stride(strides, what: str) -> int:
    found = {s for s in strides if s}
    if len(found) > 1:
        raise ValueError(f"{what} must share one row stride")
    return found.pop() if found else 0


class KvCache:
    """A KV cache that calls write to: pools [pages, page rows, KV heads, D]
    (KV_LAYOUT_BNBSH) or [pages, KV heads, page rows, D] (KV_LAYOUT_BNNBSD)
    with an int32 block table [B, max pages], or contiguous tensors [B, S, KV
    heads, D]; bf16, or E4M3 codes (uint8 or float8_e4m3fn) with fp32 scales
    [pages or B, KV heads, rows, D/64], or MXFP4: bytes of two E2M1 codes (uint8,
    D/2 in the place of D; a tensor of float4_e2m1fn_x2 as .view(torch.uint8)) with E8M0
    scales (uint8 or float8_e8m0fnu) [pages or B, KV heads, rows, D/32]."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_table: Optional[torch.Tensor] = None, *,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 kv_layout: int = _abi.KV_LAYOUT_BNBSH):
        if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
            raise ValueError("k_cache and v_cache must be 4-d and alike")
        head_major = kv_layout == _abi.KV_LAYOUT_BNNBSD
        n, rows, heads, dim = (int(x) for x in k_cache.shape)
        if head_major:
            rows, heads = heads, rows
        coded = k_cache.dtype in (torch.uint8, torch.float8_e4m3fn)
        if not coded and k_cache.dtype != torch.bfloat16:
            raise ValueError("a cache is bfloat16, E4M3 codes (uint8, float8_e4m3fn) or bytes of "
                             "two E2M1 codes (uint8)")
        if coded and (k_scale is None or v_scale is None):
            raise ValueError("an FP8 or MXFP4 cache needs k_scale and v_scale")
        if not coded and (k_scale is not None or v_scale is not None):
            raise ValueError("scales belong to an FP8 or MXFP4 cache")
        # (both hold bytes: the type of the scales tells them apart)
        mx = k_cache.dtype == torch.uint8 and k_scale.dtype in (torch.uint8, torch.float8_e8m0fnu)
        dim = 2 * dim if mx else dim
        self.device = k_cache.device
        self.num_kv_heads, self.head_dim = heads, dim
        self.tensors = (k_cache, v_cache, block_table, k_scale, v_scale)  # kept alive
        c = self.params = _abi.KvCacheParams()
        c.num_kv_heads, c.head_dim, c.kv_layout = heads, dim, kv_layout
        c.k_cache, c.v_cache = _ptr(_contig(k_cache, "k_cache")), _ptr(_contig(v_cache, "v_cache"))
        if v_cache.device != self.device:
            raise ValueError("k_cache and v_cache must be on one device")
        c.kv_dtype = _abi.KV_MXFP4 if mx else _abi.KV_FP8_E4M3 if coded else _abi.KV_BF16
        if coded:
            c.quant_tile = 32 if mx else 64
            shape = (n, heads, rows, dim // c.quant_tile)
            dtype = k_scale.dtype if mx else torch.float32
            c.k_scale = _checked(k_scale, "k_scale", dtype, shape, self.device)
            c.v_scale = _checked(v_scale, "v_scale", dtype, shape, self.device)
        if block_table is None:
            self.batch, self.capacity = n, rows
            c.max_seqlen_kv = rows
        else:
            if block_table.dim() != 2:
                raise ValueError("block_table must be [B, max pages]")
            self.batch, pages = (int(x) for x in block_table.shape)
            self.capacity = pages * rows
            c.block_table = _checked(block_table, "block_table", torch.int32, (self.batch, pages),
                                     self.device)
            c.max_blocks_per_seq, c.block_size, c.num_blocks = pages, rows, n
        c.batch = self.batch

    def _lens(self, t, name):
        return _checked(t, name, torch.int32, (self.batch,), self.device)

    def _state(self, t, name, dtype):
        return _state(t, name, dtype, self.batch, self.num_kv_heads, self.capacity, self.device)


class KvAppendCall:
    """fia_kv_append with its buffers: the new rows k_new, v_new (bf16 [B, S, KV
    heads, D], or [T, KV heads, D] with cu_seqlens_q) go behind the keys of their
    sequences; `seqused_kv` holds the lengths with the new rows, as the attention
    after it takes them.  Tokens may be strided (a slice of a fused projection).
    `weights` (fp32) and `positions` (int32), [B, KV heads, >= capacity], get 0
    and the tokens' places; `status` (int32 [1]) becomes 3 if a row had no place."""

    def __init__(self, cache: KvCache, k_new: torch.Tensor, v_new: torch.Tensor,
                 seqused_kv: torch.Tensor, *, cu_seqlens_q: Optional[torch.Tensor] = None,
                 weights: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 tokens_seen: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None):
        self.cache = cache
        self.tensors = (k_new, v_new, seqused_kv, cu_seqlens_q, weights, positions, tokens_seen,
                        status)
        if k_new.shape != v_new.shape or k_new.dim() != (4 if cu_seqlens_q is None else 3):
            raise ValueError("k_new and v_new must be alike: [B, S, heads, D], or [T, heads, D] "
                             "with cu_seqlens_q")
        if tuple(k_new.shape[-2:]) != (cache.num_kv_heads, cache.head_dim):
            raise ValueError("k_new does not have the cache's heads")
        p = self.params = _abi.AppendParams()
        p.cache = cache.params
        if cu_seqlens_q is None:
            if k_new.shape[0] != cache.batch:
                raise ValueError("k_new does not have the cache's batch")
            p.layout, p.seqlen_q = _abi.LAYOUT_BSND, int(k_new.shape[1])
        else:
            p.layout, p.total_q = _abi.LAYOUT_TND, int(k_new.shape[0])
            p.cu_seqlens_q = _checked(cu_seqlens_q, "cu_seqlens_q", torch.int32,
                                      (cache.batch + 1,), cache.device)
        for name, t in (("k", k_new), ("v", v_new)):
            if t.dtype != torch.bfloat16 or t.device != cache.device:
                raise ValueError(f"{name}_new must be bfloat16 on the cache's device")
            setattr(p, name + "_new", _ptr(t))
            setattr(p, name + "_token_stride", self._token_stride(t, name + "_new"))
        p.seqused_kv = cache._lens(seqused_kv, "seqused_kv")
        p.tokens_seen = cache._lens(tokens_seen, "tokens_seen")
        if seqused_kv is None:
            raise ValueError("seqused_kv is required")
        p.weights, s1 = cache._state(weights, "weights", torch.float32)
        p.positions, s2 = cache._state(positions, "positions", torch.int32)
        p.state_stride = _one_stride((s1, s2), "weights and positions")
        p.status = _checked(status, "status", torch.int32, (1,), cache.device)

    @staticmethod
    def _token_stride(t: torch.Tensor, name: str) -> int:
        """Elements between tokens: rows of heads are whole, tokens evenly spaced."""
        heads, dim = int(t.shape[-2]), int(t.shape[-1])
        tok = t.dim() - 3
        n = int(t.shape[tok])
        if t.numel() == 0:
            return 0
        if (dim > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != dim):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        step = int(t.stride(tok)) if n > 1 else heads * dim
        if t.dim() == 4 and t.shape[0] > 1:
            if n == 1:
                step = int(t.stride(0))
            elif t.stride(0) != n * step:
                raise ValueError(f"{name}: tokens must be evenly spaced")
        if step < heads * dim:
            raise ValueError(f"{name}: its tokens overlap")
        return step

    def run(self, stream=None):
        _launch(self.cache.device, stream, _abi.fia_kv_append, self.params)


def kv_append(cache: KvCache, k_new: torch.Tensor, v_new: torch.Tensor, seqused_kv: torch.Tensor,
              *, stream=None, **kw):
    """Write the K and V rows of new tokens to the cache (KvAppendCall's
    arguments)."""
    KvAppendCall(cache, k_new, v_new, seqused_kv, **kw).run(stream)


class AssignPagesCall:
    """fia_assign_pages with its buffers: the pages of a paged cache brought up to the
    lengths `seqused_kv` (int32 [B], the new rows counted).  `block_table` [B, max pages]
    and `free_pages` [pages of the pool] are changed in place; `pages_held` [B] and
    `free_count` [1] give how many pages each sequence holds and how many are free, and
    become `pages_held_out` and `free_count_out` (by default: themselves).  The new rows
    are T tokens with `cu_seqlens_q` (T from `slots`, `positions` or `total_q`), else
    `seqlen_q` for every sequence; run() returns (slots, positions), int32 [T], new
    tensors unless given (None without rows): where each token goes in the pool, and its
    position.  `tokens_seen` (int32 [B]) counts the sequences' tokens where slots are no
    positions.  `status` (int32 [1]) becomes 3 where a page was missing.  New tensors are
    made on the stream that is current where the call is."""

    def __init__(self, block_table: torch.Tensor, pages_held: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, seqused_kv: torch.Tensor, *,
                 block_size: int, cu_seqlens_q: Optional[torch.Tensor] = None, seqlen_q: int = 0,
                 total_q: Optional[int] = None, tokens_seen: Optional[torch.Tensor] = None,
                 slots: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 pages_held_out: Optional[torch.Tensor] = None,
                 free_count_out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None):
        if block_table.dim() != 2 or free_pages.dim() != 1:
            raise ValueError("block_table must be [B, max pages], free_pages [pages]")
        dev = self.device = block_table.device
        batch, pages = (int(x) for x in block_table.shape)

        def ints(t, name, n):
            return _checked(t, name, torch.int32, (n,), dev)

        for name, t in (("pages_held", pages_held), ("free_count", free_count),
                        ("seqused_kv", seqused_kv)):
            if t is None:
                raise ValueError(f"{name} is required")
        p = self.params = _abi.PagesParams()
        p.batch, p.max_blocks_per_seq = batch, pages
        p.block_size, p.num_blocks = _int32(block_size, "block_size"), int(free_pages.numel())
        p.block_table = _checked(block_table, "block_table", torch.int32, (batch, pages), dev)
        p.free_pages = ints(free_pages, "free_pages", p.num_blocks)
        p.seqused_kv, p.tokens_seen = ints(seqused_kv, "seqused_kv", batch), ints(
            tokens_seen, "tokens_seen", batch)
        p.pages_held, p.free_count = ints(pages_held, "pages_held", batch), ints(
            free_count, "free_count", 1)
        self.pages_held_out = pages_held if pages_held_out is None else pages_held_out
        self.free_count_out = free_count if free_count_out is None else free_count_out
        p.pages_held_out = ints(self.pages_held_out, "pages_held_out", batch)
        p.free_count_out = ints(self.free_count_out, "free_count_out", 1)
        if cu_seqlens_q is None:
            p.layout, p.seqlen_q = _abi.LAYOUT_BSND, _int32(seqlen_q, "seqlen_q")
            rows = batch * p.seqlen_q
        else:
            given = [int(t.numel()) for t in (slots, positions) if t is not None]
            rows = given[0] if total_q is None and given else total_q
            if rows is None:
                raise ValueError("total_q is required without slots and positions")
            p.layout, p.total_q = _abi.LAYOUT_TND, _int32(rows, "total_q")
            p.cu_seqlens_q = ints(cu_seqlens_q, "cu_seqlens_q", batch + 1)
        if rows > 0 and slots is None:
            slots = torch.empty(rows, dtype=torch.int32, device=dev)
        if rows > 0 and positions is None:
            positions = torch.empty(rows, dtype=torch.int32, device=dev)
        self.slots, self.positions = slots, positions
        p.slots, p.positions = ints(slots, "slots", max(rows, 0)), ints(positions, "positions",
                                                                        max(rows, 0))
        p.status = ints(status, "status", 1)
        self.tensors = (block_table, pages_held, free_pages, free_count, seqused_kv, cu_seqlens_q,
                        tokens_seen, status)

    def run(self, stream=None):
        _launch(self.device, stream, _abi.fia_assign_pages, self.params)
        return self.slots, self.positions


def assign_pages(block_table: torch.Tensor, pages_held: torch.Tensor, free_pages: torch.Tensor,
                 free_count: torch.Tensor, seqused_kv: torch.Tensor, *, stream=None, **kw):
    """Bring a cache's pages up to its lengths (AssignPagesCall's arguments); returns
    (slots, positions), made on `stream`."""
    with _made_on(stream, block_table.device):
        return AssignPagesCall(block_table, pages_held, free_pages, free_count, seqused_kv,
                               **kw).run(stream)


class NormRopeAppendCall:
    """fia_norm_rope_append with its buffers: the heads of q and k_new normed (x * weight /
    sqrt(mean x^2 + eps), where there is a weight, bf16 [D]) and rotated to `positions`
    (int32 [T]) by `cos_sin` (fp32 [max positions, rotary dim], cosines then sines; None:
    no rotation; `interleaved`: neighbours are pairs, else halves of the rotary
    dimension), the queries to `q_out` (bf16, a new tensor unless given; may be q), k_new
    and v_new to `slots` (int32 [T]) of the cache.  q, k_new, v_new are bf16 [T, heads,
    D] or [B, S, heads, D], and tokens may be strided (slices of a fused projection).
    Rows with a position below 0 are left out; `status` (int32 [1]) becomes 3 where a
    slot or a position lies outside.  Slots differ from each other.  Weights and positions
    of a bounded cache are not set: there KvAppendCall takes the new rows.  run() returns
    q_out."""

    def __init__(self, cache: KvCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                 slots: torch.Tensor, positions: torch.Tensor,
                 cos_sin: Optional[torch.Tensor] = None, *,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
        self.cache = cache
        if k_new.shape != v_new.shape or q.dim() not in (3, 4) or k_new.dim() != q.dim() \
                or q.shape[:-2] != k_new.shape[:-2]:
            raise ValueError("q, k_new and v_new must have the same tokens: [T, heads, D] or "
                             "[B, S, heads, D]")
        if tuple(k_new.shape[-2:]) != (cache.num_kv_heads, cache.head_dim) \
                or q.shape[-1] != cache.head_dim:
            raise ValueError("k_new does not have the cache's heads")
        self.q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
        if self.q_out.shape != q.shape:
            raise ValueError(f"q_out must be {tuple(q.shape)}")
        p = self.params = _abi.NormRopeParams()
        p.cache = cache.params
        p.tokens, p.num_q_heads = math.prod(q.shape[:-2]), int(q.shape[-2])
        for name, t in (("q", q), ("k", k_new), ("v", v_new), ("q_out", self.q_out)):
            if t.dtype != torch.bfloat16 or t.device != cache.device:
                raise ValueError(f"{name} must be bfloat16 on the cache's device")
            setattr(p, name, _ptr(t))
            setattr(p, name + "_token_stride", KvAppendCall._token_stride(t, name))
        for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
            setattr(p, name, _checked(t, name, torch.bfloat16, (cache.head_dim,), cache.device))
        p.eps, p.interleaved = eps, int(interleaved)
        if cos_sin is not None:
            if cos_sin.dim() != 2:
                raise ValueError("cos_sin must be [max positions, rotary dim]")
            p.max_positions, p.rotary_dim = (int(x) for x in cos_sin.shape)
            p.cos_sin = _checked(cos_sin, "cos_sin", torch.float32, cos_sin.shape, cache.device)
        for name, t in (("slots", slots), ("positions", positions)):
            setattr(p, name, _checked(t, name, torch.int32, (p.tokens,), cache.device))
        p.status = _checked(status, "status", torch.int32, (1,), cache.device)
        self.tensors = (q, k_new, v_new, slots, positions, cos_sin, q_weight, k_weight, status)

    def run(self, stream=None):
        _launch(self.cache.device, stream, _abi.fia_norm_rope_append, self.params)
        return self.q_out


def norm_rope_append(cache: KvCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                     slots: torch.Tensor, positions: torch.Tensor,
                     cos_sin: Optional[torch.Tensor] = None, *, stream=None, **kw):
    """Norm and rotate the heads of new tokens and write K and V to their slots
    (NormRopeAppendCall's arguments); returns q_out, made on `stream`."""
    with _made_on(stream, cache.device):
        return NormRopeAppendCall(cache, q, k_new, v_new, slots, positions, cos_sin,
                                  **kw).run(stream)


class KeyWeightsCall(FiaCall):
    """An FIA call that also adds up the attention weight of every cached key:
    weights_out = weights + this call's probabilities summed over the query rows
    and the heads of a KV head (fp32 [B, KV heads, >= capacity]).  `weights` None
    starts from zero; `weights_out` defaults to a new tensor of zeros, and may be
    `weights` itself.  run() returns (out, lse, weights_out)."""

    def __init__(self, prob, weights: Optional[torch.Tensor] = None,
                 weights_out: Optional[torch.Tensor] = None, num_sms: int = 0, out=None, lse=None):
        dev = self.device = prob.q.device
        self.prob = prob
        self.out, self.lse = _outputs(prob, out, lse, True)
        self.params = params_from_problem(prob, self.out, self.lse, num_sms)
        capacity = int(prob.S_kv if prob.block_table is None
                       else prob.block_table.shape[1] * prob.block_size)
        self.weights = weights
        self.weights_out = (_new_state(weights, torch.float32, prob.B, prob.KVN, capacity, dev)
                            if weights_out is None else weights_out)
        w = self.weights_params = _abi.WeightsParams()
        w.weights_in, s1 = _state(weights, "weights", torch.float32, prob.B, prob.KVN, capacity,
                                  dev)
        w.weights_out, s2 = _state(self.weights_out, "weights_out", torch.float32, prob.B,
                                   prob.KVN, capacity, dev)
        w.state_stride = _one_stride((s1, s2), "weights and weights_out")
        with _on(dev):
            self.ws_bytes = _abi.fia_get_weights_workspace_size(self.params, w)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def execute(self, stream=None):
        _launch(self.device, stream, _abi.fia_execute_weights, self.params, self.weights_params,
                self.ws.data_ptr(), self.ws_bytes)

    def run(self, stream=None):
        _launch(self.device, stream, _abi.fia_run_weights, self.params, self.weights_params,
                self.ws.data_ptr(), self.ws_bytes)
        return self.out, self.lse, self.weights_out


class KvEvictCall:
    """fia_kv_evict with its buffers and workspace: every KV head of a sequence
    with more than `budget` keys keeps `budget` of them -- positions below
    `first_tokens`, the newest `recent_tokens`, then the largest `weights` (ties
    to the lowest slot) -- and the kept keys past the budget move into the evicted
    slots below it.  run() returns (seqused_out, weights_out, positions_out); the
    outputs default to new tensors, and weights_out / positions_out may be the
    inputs themselves.  seqused_out is never seqused_kv: problems and calls that hold
    the old length tensor go on with the old lengths until the new ones are copied
    into it.  New tensors and the workspace are made on the stream that is
    current where the call is: order a run on another stream behind it, and keep
    the object until that stream has run it (kv_evict takes care of both)."""

    def __init__(self, cache: KvCache, seqused_kv: torch.Tensor, weights: torch.Tensor, *,
                 budget: int, first_tokens: int = 0, recent_tokens: int = 0,
                 positions: Optional[torch.Tensor] = None,
                 tokens_seen: Optional[torch.Tensor] = None,
                 weights_out: Optional[torch.Tensor] = None,
                 positions_out: Optional[torch.Tensor] = None,
                 seqused_out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None):
        self.cache = cache
        if seqused_kv is None or weights is None:
            raise ValueError("seqused_kv and weights are required")
        self.seqused_out = torch.empty_like(seqused_kv) if seqused_out is None else seqused_out
        def new(dtype):
            return _new_state(weights, dtype, cache.batch, cache.num_kv_heads, cache.capacity,
                              cache.device)

        self.weights_out = new(torch.float32) if weights_out is None else weights_out
        if positions_out is None:
            positions_out = new(torch.int32)
        self.positions_out = positions_out
        self.tensors = (seqused_kv, weights, positions, tokens_seen, status)
        p = self.params = _abi.EvictParams()
        p.cache = cache.params
        p.seqused_kv = cache._lens(seqused_kv, "seqused_kv")
        p.seqused_out = cache._lens(self.seqused_out, "seqused_out")
        p.tokens_seen = cache._lens(tokens_seen, "tokens_seen")
        p.weights_in, s1 = cache._state(weights, "weights", torch.float32)
        p.weights_out, s2 = cache._state(self.weights_out, "weights_out", torch.float32)
        p.positions_in, s3 = cache._state(positions, "positions", torch.int32)
        p.positions_out, s4 = cache._state(positions_out, "positions_out", torch.int32)
        p.state_stride = _one_stride((s1, s2, s3, s4), "weights and positions")
        p.budget = _int32(budget, "budget")
        p.first_tokens = _int32(first_tokens, "first_tokens")
        p.recent_tokens = _int32(recent_tokens, "recent_tokens")
        p.status = _checked(status, "status", torch.int32, (1,), cache.device)
        self.ws_bytes = _abi.fia_get_evict_workspace_size(p)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=cache.device)

    def run(self, stream=None):
        _launch(self.cache.device, stream, _abi.fia_kv_evict, self.params, self.ws.data_ptr(),
                self.ws_bytes)
        return self.seqused_out, self.weights_out, self.positions_out


def kv_evict(cache: KvCache, seqused_kv: torch.Tensor, weights: torch.Tensor, *, stream=None,
             **kw):
    """Cut the cache down to a budget (KvEvictCall's arguments); returns
    (seqused_out, weights_out, positions_out), made on `stream`."""
    with _made_on(stream, cache.device):
        return KvEvictCall(cache, seqused_kv, weights, **kw).run(stream)


# ----------------------------------------------------------------------------
# sparse shared-KV attention
# ----------------------------------------------------------------------------

def sparse_params_from_problem(sp, out: torch.Tensor, lse: Optional[torch.Tensor],
                               num_sms: int = 0) -> SparseParams:
    p = SparseParams()
    p.batch, p.num_q_heads, p.head_dim, p.layout = sp.B, sp.N1, sp.D, sp.layout
    p.max_seqlen_q, p.total_q = sp.S1, sp.T1
    p.q, p.out, p.lse = _ptr(sp.q), _ptr(out), _ptr(lse)
    p.ori_kv, p.ori_block_table = _ptr(sp.ori_kv), _ptr(sp.ori_block_table)
    p.ori_max_blocks = int(sp.ori_block_table.shape[1])
    p.ori_block_size, p.ori_num_blocks = sp.ori_block_size, int(sp.ori_kv.shape[0])
    p.cmp_kv, p.cmp_block_table = _ptr(sp.cmp_kv), _ptr(sp.cmp_block_table)
    p.cmp_max_blocks = 0 if sp.cmp_block_table is None else int(sp.cmp_block_table.shape[1])
    p.cmp_block_size = sp.cmp_block_size if sp.cmp_kv is not None else 0
    p.cmp_num_blocks = 0 if sp.cmp_kv is None else int(sp.cmp_kv.shape[0])
    p.topk = sp.K2
    p.cmp_sparse_indices = _ptr(sp.cmp_sparse_indices)
    p.cu_seqlens_q, p.seqused_kv, p.sinks = _ptr(sp.cu_seqlens_q), _ptr(sp.seqused_kv), _ptr(
        sp.sinks)
    p.softmax_scale = sp.scale
    p.cmp_ratio = sp.cmp_ratio if sp.cmp_kv is not None else 1
    p.ori_win_left, p.ori_win_right = sp.win_left, sp.win_right
    p.num_sms = num_sms
    p.kv_dtype = getattr(sp, "kv_dtype", _abi.SPARSE_KV_BF16)
    if p.kv_dtype == _abi.SPARSE_KV_FP8_PACKED:
        p.tile_size, p.rope_head_dim = 64, 64
    return p


class SparseCall:
    """Metadata + main call of the shared-KV sparse attention."""

    def __init__(self, sp, with_lse: bool = True, num_sms: int = 0):
        dev = sp.q.device
        self.sp = sp
        self.out = torch.empty_like(sp.q)
        self.lse = (torch.empty((sp.rows, sp.N1), dtype=torch.float32, device=dev)
                    if with_lse else None)
        self.params = sparse_params_from_problem(sp, self.out, self.lse, num_sms)
        self.metadata = torch.zeros(1024, dtype=torch.int32, device=dev)
        self.ws = None
        self.ws_bytes = 0

    def plan(self, stream=None):
        n = _launch(self.out.device, stream, _abi.sparse_attn_metadata, self.params,
                    self.metadata.data_ptr())
        if self.ws is None or self.ws.numel() < n:
            self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.out.device)
        self.ws_bytes = n

    def run(self, stream=None):
        if self.ws is None:
            self.plan(stream)
        _launch(self.out.device, stream, _abi.sparse_attn_run, self.params,
                self.metadata.data_ptr(), self.ws.data_ptr(), self.ws_bytes)
        return self.out, self.lse


# ----------------------------------------------------------------------------
# log-sum-exp combine of partial results (context parallelism over the keys)
# ----------------------------------------------------------------------------

def lse_combine(outs, lses, *, layout: int, num_heads: int, batch: int = 0, seqlen_q: int = 0,
                total_q: int = 0, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, sinks: Optional[torch.Tensor] = None,
                stream=None):
    """Combine results of the same query rows against disjoint key sets with
    fia_lse_combine.  `outs` are bf16 tensors in the FIA out layout, `lses`
    the matching fp32 lse tensors, computed without sinks; `sinks` (fp32
    [num_heads]) enter here, once.  Returns (out, lse)."""
    import ctypes
    n = len(outs)
    if n != len(lses) or not 1 <= n <= _abi.COMBINE_MAX_PARTS:
        raise ValueError("one lse per part, 1..16 parts")
    for t in list(outs) + list(lses):
        _contig(t, "part")
    out = torch.empty_like(outs[0]) if out is None else out
    lse = torch.empty_like(lses[0]) if lse is None else lse
    c = _abi.CombineParams()
    c.n_parts, c.layout, c.batch, c.seqlen_q, c.total_q = n, layout, batch, seqlen_q, total_q
    c.num_heads, c.head_dim = num_heads, int(outs[0].shape[-1])
    o_arr = (ctypes.c_void_p * n)(*[_ptr(t) for t in outs])
    l_arr = (ctypes.c_void_p * n)(*[_ptr(t) for t in lses])
    c.o_parts = ctypes.cast(o_arr, ctypes.POINTER(ctypes.c_void_p))
    c.lse_parts = ctypes.cast(l_arr, ctypes.POINTER(ctypes.c_void_p))
    c.out, c.lse, c.sinks = _ptr(out), _ptr(lse), _ptr(sinks)
    _launch(out.device, stream, _abi.fia_lse_combine, c)
    return out, lse
