"""The paged key/value cache: appending to it and attending to it (``fa_kv_append*``, ``fa_fwd_paged*``).

Pools are CUDA tensors [n_pages, Hkv, page_size, d], bf16 or float8_e4m3fn; e4m3 pools go with fp32
scales [n_pages, Hkv].  Key j of sequence b is row j % page_size of page page_table[b, j // page_size].
``key_lens[b]`` counts sequence b's keys after this step's append, ``new_lens[b]`` (all Nq by default)
its new ones, so that one step is

    q = kv_append(k, v, k_cache, v_cache, page_table, key_lens, new_lens, rope=rope_tables(...), q=q)
    o, lse = attention_paged(q, k_cache, v_cache, page_table, key_lens, causal=True, new_lens=new_lens)

Both calls run on the current stream of the pools' device, and can be captured into a CUDA graph whose
replays read the lengths and the table anew.  They are for serving: no gradient flows through them.
"""
import functools

import torch

from . import _lib


@functools.cache
def _binding():
    """The compiled argument marshalling (csrc/paged_binding.cpp): it checks, allocates and calls, and returns None where
    something does not fit, which the functions here then name."""
    _lib.load()
    try:
        from . import _paged
    except ImportError as e:
        raise RuntimeError("the compiled module exact_io_aware_68_b200/_paged.so is missing or does not load: build it with "
                           f"`python -m exact_io_aware_68_b200.build` (there is no fallback): {e}") from e
    return _paged


def _failed(status):
    return _lib.FAError(status, _lib.load().fa_get_error().decode())


def _need(ok, text):
    if not ok:
        raise ValueError(text)


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
        _need(all(n == 1 or st == want for n, st, want in zip(shape[1:], t.stride()[1:], (shape[2] * d, d, 1))),
              f"{name} must be contiguous within a page")
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


def _need_tensor(name, t, dtype, shape, device):
    _need(t is None or (t.device == device and t.dtype == dtype and t.is_contiguous() and t.shape == shape),
          f"{name} must be contiguous {dtype} {tuple(shape)} on {device}")


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
    the scales of e4m3 pools) in place; returns the rotated queries, contiguous [B, Hq, Nq, d], or None.  q_out: where
    to write those; a contiguous q itself, or no memory of q's, k's or v's."""
    cos, sin = (None, None) if rope is None else rope
    out = _binding().append(k, v, k_cache, v_cache, page_table, key_lens, new_lens, cos, sin, interleaved, q, k_scale, v_scale, q_out)
    if out is True:
        return None
    if type(out) is int:
        raise _failed(out)
    if out is not None:
        return out
    # something does not fit
    _need(k.dim() == 4 and v.shape == k.shape, f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [B, Hkv, Nq, d], both the same")
    B, Hkv, Nq, d = k.shape
    _refuse_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d)
    device = k_cache.device
    _need(k_cache.shape[1] == Hkv, f"the pools have {k_cache.shape[1]} heads, k has {Hkv}")
    _need(q is None or (q.dim() == 4 and q.shape[0] == B and q.shape[2:] == k.shape[2:]),
          f"q has shape {tuple(q.shape) if q is not None else None}, expected ({B}, Hq, {Nq}, {d})")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            continue
        _need(t.device == device, f"{name} is on {t.device}, k_cache on {device}")
        _need(t.dtype == torch.bfloat16, f"{name} must be torch.bfloat16, got {t.dtype}")
        _need(t.stride(3) == 1, f"{name} must be contiguous in its last dimension")
    _need((cos is None) == (sin is None), "rope needs both tables, (cos, sin)")
    for name, t in (("rope cos", cos), ("rope sin", sin)):
        _need(t is None or (t.dim() == 2 and t.dtype == torch.float32 and t.is_contiguous() and t.device == device and t.shape == cos.shape),
              f"{name} must be contiguous fp32 [max_pos, rot / 2] on {device}, cos and sin alike")
    _need(q_out is None or q is not None, "q_out goes with q")
    if q is not None:
        _need_tensor("q_out", q_out, torch.bfloat16, q.shape, device)
    raise ValueError("the arguments of kv_append do not fit one another")


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
    key_lens[b] - new_lens[b] + i; causal keeps the keys up to it.  Queries i >= new_lens[b] get O = 0, lse = -inf.
    o must not overlap q."""
    out = _binding().attention(q, k_cache, v_cache, page_table, key_lens, new_lens, k_scale, v_scale, workspace, o, lse, scale, causal)
    if type(out) is tuple:
        return out
    if out is not None:
        raise _failed(out)
    # something does not fit
    _need(q.dim() == 4, f"q has shape {tuple(q.shape)}, expected [B, Hq, Nq, d]")
    B, Hq, Nq, d = q.shape
    _refuse_cache(k_cache, v_cache, k_scale, v_scale, page_table, key_lens, new_lens, B, d)
    device = k_cache.device
    _need_tensor("q", q, torch.bfloat16, q.shape, device)
    _need_tensor("o", o, torch.bfloat16, q.shape, device)
    _need_tensor("lse", lse, torch.float32, q.shape[:3], device)
    _need(workspace is None or (workspace.dtype == torch.uint8 and workspace.is_contiguous() and workspace.device == device),
          f"workspace must be contiguous uint8 on {device}")
    raise ValueError("the arguments of attention_paged do not fit one another")
