"""The paged key/value cache: appending to it and attending to it (``fa_kv_append*``, ``fa_fwd_paged*``).

Pools are CUDA tensors [n_pages, Hkv, page_size, d], bf16 or float8_e4m3fn; e4m3 pools go with fp32
scales [n_pages, Hkv].  Key j of sequence b is row j % page_size of page page_table[b, j // page_size].
``key_lens[b]`` counts sequence b's keys after this step's append, ``new_lens[b]`` (all Nq by default)
its new ones, so that one step is

    q = kv_append(k, v, k_cache, v_cache, page_table, key_lens, new_lens, rope=rope_tables(...), q=q)
    o, lse = attention_paged(q, k_cache, v_cache, page_table, key_lens, causal=True, new_lens=new_lens)

Both calls run on the current stream of the pools' device, and can be captured into a CUDA graph whose
replays read the lengths and the table anew.
"""
import ctypes
import functools
import math

import torch

from . import _lib

_STRIDES = ctypes.c_int64 * 9


def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _cache_fits(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d, dev):
    """Whether the cache's tensors fit one another: the quick form of ``_refuse_cache``, which says what does not."""
    shape, dt = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or dev < 0:
        return False
    n_pages, heads, page, dd = shape
    inner = (page * d, d, 1)
    if dd != d or v_cache.shape != shape or v_cache.dtype is not dt or k_cache.stride()[1:] != inner or v_cache.stride()[1:] != inner \
            or v_cache.get_device() != dev:
        return False
    if dt is torch.float8_e4m3fn:
        pages = (n_pages, heads)
        if k_scale is None or v_scale is None or not (_fits(k_scale, torch.float32, pages, dev) and _fits(v_scale, torch.float32, pages, dev)):
            return False
    elif dt is not torch.bfloat16 or k_scale is not None or v_scale is not None:
        return False
    i32, rows = torch.int32, (B,)
    return (_fits(key_lens, i32, rows, dev) and (new_lens is None or _fits(new_lens, i32, rows, dev)) and page_table.dtype is i32
            and page_table.dim() == 2 and page_table.shape[0] == B and page_table.is_contiguous() and page_table.get_device() == dev)


def _refuse_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d):
    """Raises for the first of the cache's tensors that does not fit."""
    dev, dt, shape = k_cache.device, k_cache.dtype, tuple(k_cache.shape)
    _need(k_cache.is_cuda, "k_cache must be a CUDA tensor")
    fp8 = dt == torch.float8_e4m3fn
    _need(fp8 or dt == torch.bfloat16, f"k_cache must be bfloat16 or float8_e4m3fn, got {dt}")
    _need(len(shape) == 4 and tuple(v_cache.shape) == shape, f"k_cache {shape} and v_cache {tuple(v_cache.shape)} must be "
          "[n_pages, Hkv, page_size, d], both the same")
    _need(shape[3] == d, f"the pools have d = {shape[3]}, the heads {d}")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t.stride()[1:] == (shape[2] * d, d, 1), f"{name} must be contiguous within a page")
    _need((k_scale is not None) == fp8 and (v_scale is not None) == fp8, "k_scale and v_scale go with float8_e4m3fn pools")
    for name, t, dtype, sh in (("v_cache", v_cache, dt, shape), ("k_scale", k_scale, torch.float32, shape[:2]),
                               ("v_scale", v_scale, torch.float32, shape[:2]), ("key_lens", key_lens, torch.int32, (B,)),
                               ("new_lens", new_lens, torch.int32, (B,)), ("page_table", page_table, torch.int32, None)):
        if t is None:
            continue
        _need(t.device == dev, f"{name} is on {t.device}, k_cache on {dev}")
        _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
        _need(name == "v_cache" or t.is_contiguous(), f"{name} must be contiguous")
        _need(sh is None or tuple(t.shape) == sh, f"{name} has shape {tuple(t.shape)}, expected {sh}")
    _need(page_table.dim() == 2 and page_table.shape[0] == B, f"page_table has shape {tuple(page_table.shape)}, expected "
          f"({B}, max_pages)")
    raise ValueError("the tensors of the cache do not fit one another")


def _fits(t, dtype, shape, dev):
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev


@functools.cache
def _entry(name):
    return getattr(_lib.load(), name)


def _call(dev, name, *args):
    """The entry point on the current stream of device `dev`, with that device current for the call."""
    if dev == torch._C._cuda_getDevice():
        status = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise _lib.FAError(status, _lib.load().fa_get_error().decode())


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(B, Hq, Hkv, Nq, d, dev):
    with torch.cuda.device(dev):
        return _lib.load().fa_fwd_paged_workspace_size(B, Hq, Hkv, Nq, d)


def rope_tables(max_pos, rot_dim, base=10000.0, device="cuda"):
    """(cos, sin) fp32 [max_pos, rot_dim / 2] of the angles position * base^(-2 i / rot_dim), formed in fp64."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def kv_append(k, v, k_cache, v_cache, page_table, key_lens, new_lens=None, rope=None, interleaved=False, q=None, k_scale=None,
              v_scale=None, q_out=None):
    """Append this step's keys and values to the pools (``fa_kv_append``, ``fa_kv_append_e4m3``).

    k, v: bf16 [B, Hkv, Nq, d]; q: bf16 [B, Hq, Nq, d] or None; any strides that are multiples of 8 with d
    contiguous (views of a projection's output need no copy).  rope: (cos, sin) tables, applied to k and q by position
    (``rope_tables``); interleaved: pairs (2i, 2i + 1) instead of (i, i + rot / 2).  Writes the pools (and
    the scales of e4m3 pools) in place; returns the rotated queries, contiguous [B, Hq, Nq, d], or None."""
    if k.dim() != 4 or v.shape != k.shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [B, Hkv, Nq, d], both the same")
    B, Hkv, Nq, d = k.shape
    dev = k_cache.get_device()
    if not _cache_fits(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d, dev):
        _refuse_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d)
    n_pages, heads, page, _ = k_cache.shape
    if heads != Hkv:
        raise ValueError(f"the pools have {heads} heads, k has {Hkv}")
    bf16 = torch.bfloat16
    Hq = Hkv
    if q is not None:
        qs = q.shape
        if len(qs) != 4 or qs[0] != B or qs[2] != Nq or qs[3] != d:
            raise ValueError(f"q has shape {tuple(qs)}, expected ({B}, Hq, {Nq}, {d})")
        Hq = qs[1]
    strides = []
    for t in (q, k, v):
        if t is None:
            strides += (0, 0, 0)
            continue
        if t.get_device() != dev or t.dtype is not bf16 or t.stride(3) != 1:
            name = "q" if t is q else "k" if t is k else "v"
            _need(t.device == k_cache.device, f"{name} is on {t.device}, k_cache on {k_cache.device}")
            _need(t.dtype is bf16, f"{name} must be torch.bfloat16, got {t.dtype}")
            raise ValueError(f"{name} must be contiguous in its last dimension")
        b, h, n, _ = t.stride()
        # the stride of a dimension of size one is never taken
        strides += (b if B > 1 else 0, h if t.shape[1] > 1 else 0, n if Nq > 1 else 0)
    cos = sin = None
    max_pos = rot = 0
    if rope is not None:
        cos, sin = rope
        for name, t in (("rope cos", cos), ("rope sin", sin)):
            if t.dim() != 2 or not _fits(t, torch.float32, cos.shape, dev):
                raise ValueError(f"{name} must be contiguous fp32 [max_pos, rot / 2] on {k_cache.device}, cos and sin alike")
        max_pos, half = cos.shape
        rot, cos, sin = 2 * half, cos.data_ptr(), sin.data_ptr()
    if q is None:
        _need(q_out is None, "q_out goes with q")
        q_ptr = out_ptr = None
    else:
        if q_out is None:
            q_out = torch.empty_strided((B, Hq, Nq, d), (Hq * Nq * d, Nq * d, d, 1), dtype=bf16, device=k_cache.device)
        elif not _fits(q_out, bf16, q.shape, dev):
            raise ValueError(f"q_out must be contiguous bfloat16 {tuple(q.shape)} on {k_cache.device}")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    name, scales = ("fa_kv_append", ()) if k_scale is None else ("fa_kv_append_e4m3", (k_scale.data_ptr(), v_scale.data_ptr()))
    _call(dev, name, q_ptr, k.data_ptr(), v.data_ptr(), _STRIDES(*strides), out_ptr, k_cache.data_ptr(), v_cache.data_ptr(), *scales,
          k_cache.stride(0), v_cache.stride(0), page_table.data_ptr(), key_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
          cos, sin, max_pos, rot, int(bool(interleaved)), B, Hq, Hkv, Nq, d, n_pages, page, page_table.shape[1])
    return q_out


def paged_workspace(B, Hq, Hkv, Nq, d, device):
    """A workspace tensor for ``attention_paged`` (torch allocations are 256-byte aligned)."""
    device = torch.empty(0, device=device).device
    return torch.empty(_workspace_bytes(B, Hq, Hkv, Nq, d, device.index), dtype=torch.uint8, device=device)


def attention_paged(q, k_cache, v_cache, page_table, key_lens, scale=None, causal=False, new_lens=None, k_scale=None,
                    v_scale=None, workspace=None, o=None, lse=None):
    """O and lse of Nq new queries per head against their sequences' keys in the pools (``fa_fwd_paged``,
    ``fa_fwd_paged_e4m3``).

    q: bf16 [B, Hq, Nq, d] contiguous, Hq a multiple of the pools' Hkv.  Query i of sequence b stands at position
    key_lens[b] - new_lens[b] + i; causal keeps the keys up to it.  Queries i >= new_lens[b] get O = 0, lse = -inf."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q has shape {tuple(shape)}, expected [B, Hq, Nq, d]")
    B, Hq, Nq, d = shape
    dev = k_cache.get_device()
    if not _cache_fits(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d, dev):
        _refuse_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d)
    device = k_cache.device
    if not _fits(q, torch.bfloat16, shape, dev):
        raise ValueError(f"q must be contiguous bfloat16 on {device}")
    n_pages, Hkv, page, _ = k_cache.shape
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(B, Hq, Hkv, Nq, d, dev), dtype=torch.uint8, device=device)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace must be contiguous uint8 on {device}")
    if o is None:
        o = torch.empty_like(q)   # q is contiguous
    elif not _fits(o, torch.bfloat16, shape, dev):
        raise ValueError(f"o must be contiguous bfloat16 {tuple(shape)} on {device}")
    if lse is None:
        lse = torch.empty_strided((B, Hq, Nq), (Hq * Nq, Nq, 1), dtype=torch.float32, device=device)
    elif not _fits(lse, torch.float32, shape[:3], dev):
        raise ValueError(f"lse must be contiguous float32 {tuple(shape[:3])} on {device}")
    name, scales = ("fa_fwd_paged", ()) if k_scale is None else ("fa_fwd_paged_e4m3", (k_scale.data_ptr(), v_scale.data_ptr()))
    _call(dev, name, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), *scales, o.data_ptr(), lse.data_ptr(), k_cache.stride(0),
          v_cache.stride(0), page_table.data_ptr(), key_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
          B, Hq, Hkv, Nq, d, n_pages, page, page_table.shape[1], 1.0 / math.sqrt(d) if scale is None else float(scale),
          int(bool(causal)), workspace.data_ptr(), workspace.numel())
    return o, lse
