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
import math

import torch

from . import _lib

_STRIDES = ctypes.c_int64 * 9


def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _check_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d):
    """(e4m3?, device) of the pools, after the checks that both calls share."""
    dev, dt, shape = k_cache.device, k_cache.dtype, k_cache.shape
    _need(k_cache.is_cuda, "k_cache must be a CUDA tensor")
    fp8 = dt == torch.float8_e4m3fn
    _need(fp8 or dt == torch.bfloat16, f"k_cache must be bfloat16 or float8_e4m3fn, got {dt}")
    _need(v_cache.dtype == dt, f"v_cache must be {dt} like k_cache, got {v_cache.dtype}")
    _need(len(shape) == 4 and v_cache.shape == shape, f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} must be "
          "[n_pages, Hkv, page_size, d], both the same")
    n_pages, Hkv, page, dd = shape
    _need(dd == d, f"the pools have d = {dd}, the heads {d}")
    inner = (page * d, d, 1)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t.stride()[1:] == inner, f"{name} must be contiguous within a page")
    _need((k_scale is not None) == fp8 and (v_scale is not None) == fp8, "k_scale and v_scale go with float8_e4m3fn pools")
    for name, t, dtype, sh in (("v_cache", v_cache, dt, shape), ("k_scale", k_scale, torch.float32, (n_pages, Hkv)),
                               ("v_scale", v_scale, torch.float32, (n_pages, Hkv)),
                               ("key_lens", key_lens, torch.int32, (B,)), ("new_lens", new_lens, torch.int32, (B,)),
                               ("page_table", page_table, torch.int32, None)):
        if t is None:
            continue
        _need(t.device == dev, f"{name} is on {t.device}, k_cache on {dev}")
        _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
        if name != "v_cache":
            _need(t.is_contiguous(), f"{name} must be contiguous")
        _need(sh is None or t.shape == sh, f"{name} has shape {tuple(t.shape)}, expected {sh}")
    _need(page_table.dim() == 2 and page_table.shape[0] == B, f"page_table has shape {tuple(page_table.shape)}, expected "
          f"({B}, max_pages)")
    return fp8, dev


def _call(dev, name, *args):
    """The entry point on the current stream of `dev`, with that device current for the call."""
    if dev.index == torch.cuda.current_device():
        _lib.call(name, *args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            _lib.call(name, *args, torch.cuda.current_stream(dev).cuda_stream)


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
    _need(k.dim() == 4 and v.shape == k.shape, f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [B, Hkv, Nq, d], both the same")
    B, Hkv, Nq, d = k.shape
    fp8, dev = _check_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d)
    n_pages, heads, page = k_cache.shape[:3]
    _need(heads == Hkv, f"the pools have {heads} heads, k has {Hkv}")
    Hq = Hkv
    if q is not None:
        _need(q.dim() == 4 and q.shape[0] == B and q.shape[2:] == k.shape[2:], f"q has shape {tuple(q.shape)}, expected "
              f"({B}, Hq, {Nq}, {d})")
        Hq = q.shape[1]
    strides = []
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            strides += [0, 0, 0]
            continue
        _need(t.device == dev, f"{name} is on {t.device}, k_cache on {dev}")
        _need(t.dtype == torch.bfloat16, f"{name} must be torch.bfloat16, got {t.dtype}")
        st = t.stride()
        _need(st[3] == 1, f"{name} must be contiguous in its last dimension")
        # the stride of a dimension of size one is never taken
        strides += [s if n > 1 else 0 for s, n in zip(st[:3], t.shape[:3])]
    cos = sin = None
    max_pos = rot = 0
    if rope is not None:
        cos, sin = rope
        for name, t in (("rope cos", cos), ("rope sin", sin)):
            _need(t.device == dev and t.dtype == torch.float32 and t.is_contiguous() and t.dim() == 2 and t.shape == cos.shape,
                  f"{name} must be contiguous fp32 [max_pos, rot / 2] on {dev}, cos and sin alike")
        max_pos, rot = cos.shape[0], 2 * cos.shape[1]
        cos, sin = cos.data_ptr(), sin.data_ptr()
    if q is None:
        _need(q_out is None, "q_out goes with q")
    elif q_out is None:
        q_out = torch.empty((B, Hq, Nq, d), dtype=torch.bfloat16, device=dev)
    else:
        _need(q_out.device == dev and q_out.dtype == torch.bfloat16 and q_out.is_contiguous() and q_out.shape == q.shape,
              f"q_out must be contiguous bfloat16 {tuple(q.shape)} on {dev}")
    _call(dev, "fa_kv_append_e4m3" if fp8 else "fa_kv_append", None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
          _STRIDES(*strides), None if q is None else q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          *((k_scale.data_ptr(), v_scale.data_ptr()) if fp8 else ()), k_cache.stride(0), v_cache.stride(0),
          page_table.data_ptr(), key_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(), cos, sin, max_pos, rot,
          int(bool(interleaved)), B, Hq, Hkv, Nq, d, n_pages, page, page_table.shape[1])
    return q_out


def paged_workspace(B, Hq, Hkv, Nq, d, device):
    """A workspace tensor for ``attention_paged`` (torch allocations are 256-byte aligned)."""
    with torch.cuda.device(device):
        n = _lib.load().fa_fwd_paged_workspace_size(B, Hq, Hkv, Nq, d)
    return torch.empty(n, dtype=torch.uint8, device=device)


def attention_paged(q, k_cache, v_cache, page_table, key_lens, scale=None, causal=False, new_lens=None, k_scale=None,
                    v_scale=None, workspace=None, o=None, lse=None):
    """O and lse of Nq new queries per head against their sequences' keys in the pools (``fa_fwd_paged``,
    ``fa_fwd_paged_e4m3``).

    q: bf16 [B, Hq, Nq, d] contiguous, Hq a multiple of the pools' Hkv.  Query i of sequence b stands at position
    key_lens[b] - new_lens[b] + i; causal keeps the keys up to it.  Queries i >= new_lens[b] get O = 0, lse = -inf."""
    _need(q.dim() == 4, f"q has shape {tuple(q.shape)}, expected [B, Hq, Nq, d]")
    B, Hq, Nq, d = q.shape
    fp8, dev = _check_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d)
    for name, t, dtype, shape in (("q", q, torch.bfloat16, q.shape), ("o", o, torch.bfloat16, q.shape),
                                  ("lse", lse, torch.float32, q.shape[:3])):
        if t is not None:
            _need(t.device == dev and t.dtype == dtype and t.is_contiguous() and t.shape == shape,
                  f"{name} must be contiguous {dtype} {tuple(shape)} on {dev}")
    n_pages, Hkv, page = k_cache.shape[:3]
    if workspace is None:
        workspace = paged_workspace(B, Hq, Hkv, Nq, d, dev)
    else:
        _need(workspace.device == dev and workspace.dtype == torch.uint8 and workspace.is_contiguous(),
              f"workspace must be contiguous uint8 on {dev}")
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev) if lse is None else lse
    _call(dev, "fa_fwd_paged_e4m3" if fp8 else "fa_fwd_paged", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          *((k_scale.data_ptr(), v_scale.data_ptr()) if fp8 else ()), o.data_ptr(), lse.data_ptr(), k_cache.stride(0),
          v_cache.stride(0), page_table.data_ptr(), key_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
          B, Hq, Hkv, Nq, d, n_pages, page, page_table.shape[1], 1.0 / math.sqrt(d) if scale is None else float(scale),
          int(bool(causal)), workspace.data_ptr(), workspace.numel())
    return o, lse
