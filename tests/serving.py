"""The operators of a serving step over a paged cache in 64 bits, or step by step as
they are defined: MXFP4 rows, assigned pages, head norms with rotation."""
import copy
import math

import numpy as np
import torch

import fia_inputs as fi
from tests import bounded

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
KV_MXFP4 = 4


def mx_quantised(x):
    """[..., D] values (bf16, or any whose powers of two are those of float64) as bytes of
    two codes and scale bytes, from the definition: the smallest 2^e >= 2^-127 that leaves
    no magnitude over 6; the nearest code, the even one of two; infinities as the largest
    finite bf16 value, a NaN makes the scale 255 and the codes 0."""
    t = np.asarray(x.double() if isinstance(x, torch.Tensor) else x, np.float64)
    t = t.reshape(*t.shape[:-1], -1, 32)
    nan = np.isnan(t).any(-1)
    big = float(torch.finfo(torch.bfloat16).max)
    t = np.clip(np.where(nan[..., None], 0.0, t), -big, big)
    amax = np.abs(t).max(-1)
    e = np.full(amax.shape, -127)
    for k in range(-126, 128):
        e = np.where(6 * 2.0 ** (k - 1) < amax, k, e)
    e = np.where(amax > 0, e, 0)
    y = np.abs(t) / (2.0 ** e)[..., None]
    far = np.abs(y[..., None] - E2M1)
    best = far.min(-1, keepdims=True)
    code = np.where(far == best, np.arange(8) % 2 * 10 + np.arange(8) * 0.01, 99).argmin(-1)
    code = np.where(nan[..., None], 0, code + 8 * np.signbit(np.where(nan[..., None], 0.0, t)))
    scale = np.where(nan, 255, e + 127).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], -1).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def mx_values(codes, scale):
    """Bytes of two codes and scale bytes as float64 values."""
    c = codes.cpu().numpy() if isinstance(codes, torch.Tensor) else codes
    s = scale.cpu().numpy() if isinstance(scale, torch.Tensor) else scale
    c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    v = np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])
    f = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return torch.from_numpy(v * np.repeat(f, 32, -1))


def _rows(x, head_major):
    return x.permute(0, 2, 1, 3) if head_major else x


def make_mx(**kw):
    """A problem over an MXFP4 cache (its poisoned rows hold NaN scales)."""
    dev = kw.pop("device", "cpu")
    p = fi.make_fia(D=128, device="cpu", **kw)
    return as_mx(p).to(dev)


def as_mx(p):
    """The bf16 problem with its cache in MXFP4."""
    p = copy.copy(p)
    head_major = p.kv_layout == 1
    for name in "kv":
        codes, scale = mx_quantised(getattr(p, name + "_cache"))
        scale = torch.from_numpy(scale)
        setattr(p, name + "_cache", torch.from_numpy(codes))
        setattr(p, name + "_scale", (scale if head_major else scale.permute(0, 2, 1, 3)).contiguous())
    p.kv_dtype = KV_MXFP4
    return p


def decoded(p):
    """The problem with its cache as the values it stands for."""
    q = copy.copy(p.to("cpu"))
    head_major = q.kv_layout == 1
    for name in "kv":
        scale = getattr(q, name + "_scale")
        setattr(q, name + "_cache", mx_values(getattr(q, name + "_cache"),
                                              _rows(scale, not head_major).contiguous()))
        setattr(q, name + "_scale", None)
    q.kv_dtype = fi.KV_BF16
    return q


def check_mx(p, out, lse, weights=None, weights_in=None):
    """Held to the bounds of a bf16 cache: every value of the cache is one of bf16 (and of
    fp16 times a power of two), P is rounded to fp16 (decode) or bf16 (prompts); the four
    partial scores of a row and their scales round no oftener than eight steps over D."""
    bounded.check_attention(decoded(p), out, lse, weights, weights_in)


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------

def pages(table, held, free, count, lens, block, q_lens=None, cu=None, T=0, seen=None):
    """fia_assign_pages one page after another; returns (table, held, free list, count,
    slots, positions, status), the list cut to its length before the takes."""
    B, W = table.shape
    nb = len(free)
    table, free = table.copy(), list(free)
    count = min(max(count, 0), nb)
    stack, status = list(free[:count]), 0
    held = [min(max(int(h), 0), W) for h in held]
    need = [-(-min(max(int(n), 0), W * block) // block) for n in lens]
    for b in range(B):
        for k in range(need[b], held[b]):
            if len(stack) < nb:
                stack.append(int(table[b, k]))
            else:
                status = 3
    on_list = list(stack)
    out = [min(h, n) for h, n in zip(held, need)]
    for b in range(B):
        for k in range(held[b], need[b]):
            if stack:
                table[b, k] = stack.pop()
                out[b] += 1
            else:
                table[b, k], status = -1, 3
    slots, positions = np.full(T, -1), np.full(T, -1)
    if cu is None and T:
        cu = np.arange(B + 1) * (T // B)
    for b in range(B if T else 0):
        n = int(cu[b + 1]) - int(cu[b])
        for i in range(n):
            j, t = int(lens[b]) - n + i, int(cu[b]) + i
            if j < 0 or not 0 <= t < T:
                continue
            positions[t] = j if seen is None else int(seen[b]) - n + i
            page = int(table[b, j // block]) if j < W * block else -1
            if 0 <= page < nb:
                slots[t] = page * block + j % block
            else:
                status = 3
    return table, np.array(out), on_list, len(stack), slots, positions, status


# ----------------------------------------------------------------------------
# head norms and rotation
# ----------------------------------------------------------------------------

def cos_sin(positions, dim, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, dim, 2) / max(dim, 1))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def turned(x, weight, eps, table, positions, interleaved):
    """[T, heads, D] in 64 bits, normed and rotated pair by pair, and the size of the
    terms of every output (what its rounding errors go by)."""
    x = x.double().cpu()
    if weight is not None:
        x = x * weight.double().cpu() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y, size = x.clone(), x.abs()
    if table is not None and table.shape[1]:
        rot = table.shape[1]
        row = table.double().cpu()[positions.long().cpu()][:, None]
        c, s = row[..., :rot // 2], row[..., rot // 2:]
        i = torch.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size = size.clone()
        size[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        size[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, size


# fp32 steps of a normed and rotated value: the sum of D squares (products and additions,
# halved by the square root: D / 2 + 1 half steps at most), mean, eps, root and its
# inverse (four), two weights' products, two products and a sum of the rotation
def turned_tolerance(size, D):
    return (D / 2 + 12) * bounded.HALF_FP32 * size
