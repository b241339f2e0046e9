"""GB300 (sm_103a) draft-tree verify-and-accept for EAGLE-style speculative decoding.

Thin binding over the C ABI of include/eagle.h: every function marshals torch
CUDA tensors into device pointers plus the current CUDA stream and calls the
library entry point of the same name; all arithmetic runs in the library's
kernels.  PyTorch only provides device memory and streams.  Functions raise
EagleError on a non-OK status; errors found in device data are reported through
the optional ``dev_status`` int32 tensor (bits EAGLE_DEV_*).
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _lib

EAGLE_DEV_BAD_TREE = 0x01
EAGLE_DEV_BAD_TOKEN = 0x02
EAGLE_DEV_NONFINITE = 0x04
EAGLE_DEV_DEPTH = 0x08
EAGLE_DEV_CAPACITY = 0x10
EAGLE_DEV_TIMEOUT = 0x20


class EagleError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn}: {_lib.load().eagle_status_str(code).decode()} ({code})")


def lib():
    return _lib.load()


def _check(fn: str, code: int):
    if code != 0:
        raise EagleError(fn, code)


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dev_or_pinned(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    """A CUDA tensor, or a page-locked host tensor, which the GPU reads in place over
    unified addressing (the kernel then moves only the bytes it touches)."""
    if isinstance(t, torch.Tensor) and not t.is_cuda and t.is_pinned():
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t
    return _dev(t, name, dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _empty(shape, dtype, device, stream):
    """Memory that a call on `stream` writes.  It comes from that stream's pool (memory from the
    current stream's may still be in use there when another stream writes it), and the pool gets
    it back only when the current stream, where the caller goes on with it, is done with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _empty_like(t, stream):
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _status(dev_status, device):
    if dev_status is None:
        return None
    return _dev(dev_status, "dev_status", torch.int32)


# ---------------------------------------------------------------- workspace sizes
def tree_attn_workspace_size(B, n, Hq, Hkv, head_dim, Lmax) -> int:
    return int(lib().eagle_tree_attn_workspace_size(B, n, Hq, Hkv, head_dim, Lmax))


def tree_state_size(B, top_k, depth) -> int:
    return int(lib().eagle2_tree_state_size(B, top_k, depth))


# ---------------------------------------------------------------- calls
def eagle_tree_attn(q, k_cache, v_cache, kv_len, parent, scale=None, out=None, workspace=None,
                    dev_status=None, stream=None):
    """q [B,n,Hq,d], k/v cache [B,Hkv,Lmax,d] bf16; kv_len [B], parent [B,n] int32."""
    _dev(q, "q", torch.bfloat16)
    _dev(k_cache, "k_cache", torch.bfloat16)
    _dev(v_cache, "v_cache", torch.bfloat16)
    _dev(kv_len, "kv_len", torch.int32)
    _dev(parent, "parent", torch.int32)
    B, n, Hq, d = q.shape
    Hkv, Lmax = k_cache.shape[-3], k_cache.shape[-2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _dev(out, "out", torch.bfloat16)
    need = tree_attn_workspace_size(B, n, Hq, Hkv, d, Lmax)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("eagle_tree_attn", lib().eagle_tree_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(parent), _ptr(out),
        B, n, Hq, Hkv, d, Lmax, float(scale), _ptr(workspace), ws_bytes,
        _ptr(_status(dev_status, q.device)), _stream(stream)))
    return out


def eagle_ttt_attn(q, k, v, r, scale=None, out=None, dev_status=None, stream=None):
    """Training-time-test attention of the queries of round r.  q [B,S,Hq,d] and
    k / v [B,Hkv,R1,S,d] bf16 (round 0 = the original tokens); returns out [B,S,Hq,d]."""
    _dev(q, "q", torch.bfloat16)
    _dev(k, "k", torch.bfloat16)
    _dev(v, "v", torch.bfloat16)
    B, S, Hq, d = q.shape
    if k.dim() != 5 or tuple(v.shape) != tuple(k.shape) or k.shape[0] != B or k.shape[3] != S \
            or k.shape[4] != d:
        raise ValueError("eagle_ttt_attn: k / v must be [B, Hkv, R1, S, d] matching q")
    Hkv, R1 = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _dev(out, "out", torch.bfloat16)
    _check("eagle_ttt_attn", lib().eagle_ttt_attn(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, Hq, Hkv, d, R1, int(r), float(scale),
        _ptr(_status(dev_status, q.device)), _stream(stream)))
    return out


def verify_filter_workspace_size(B, n, R) -> int:
    return int(lib().eagle_verify_filter_workspace_size(B, n, R))


def eagle_d2t_inverse(d2t, V, t2d=None, dev_status=None, stream=None):
    """t2d int32 [V]: the draft id of each target id (d + d2t[d] -> d), -1 where none."""
    _dev(d2t, "d2t", torch.int32)
    t2d = _empty(V, torch.int32, d2t.device, stream) if t2d is None else t2d
    _dev(t2d, "t2d", torch.int32)
    _check("eagle_d2t_inverse", lib().eagle_d2t_inverse(
        _ptr(d2t), d2t.numel(), int(V), _ptr(t2d), _ptr(_status(dev_status, d2t.device)),
        _stream(stream)))
    return t2d


def eagle_verify_accept(target_logits, draft_logits, tokens, parent, max_depth, temperature, seed,
                        draft_row=None, accept_len=None, path=None, emit=None, row_stats=None,
                        dev_status=None, stream=None, t2d=None, top_k=0, top_p=0.0,
                        workspace=None):
    """Returns (accept_len [B], path [B,D+1], emit [B,D+1]) int32 tensors.  With t2d
    (from eagle_d2t_inverse) the draft rows are over the draft vocabulary
    [B, R, Vd] and tokens are target ids.  target_logits may be a pinned host tensor:
    the walk then reads only the rows it visits, in place."""
    _dev_or_pinned(target_logits, "target_logits", torch.float32)
    B, n, V = target_logits.shape
    R = n
    Vd = V
    if draft_logits is not None:
        _dev(draft_logits, "draft_logits", torch.float32)
        R = draft_logits.shape[1]
        Vd = draft_logits.shape[2]
    _dev(tokens, "tokens", torch.int32)
    _dev(parent, "parent", torch.int32)
    if draft_row is not None:
        _dev(draft_row, "draft_row", torch.int32)
    dev = tokens.device
    D = int(max_depth)
    accept_len = _empty(B, torch.int32, dev, stream) if accept_len is None else accept_len
    path = _empty((B, D + 1), torch.int32, dev, stream) if path is None else path
    emit = _empty((B, D + 1), torch.int32, dev, stream) if emit is None else emit
    if row_stats is not None:
        _dev(row_stats, "row_stats", torch.float32)
    if (top_k or top_p) and temperature > 0:
        if t2d is not None:
            raise ValueError("top-k / top-p filtering with a draft vocabulary is not offered")
        need = int(lib().eagle_verify_filter_workspace_size(B, n, R))
        if workspace is None:
            workspace = _empty(max(need, 1), torch.uint8, dev, stream)
        _dev(workspace, "workspace")
        _check("eagle_verify_accept_filtered", lib().eagle_verify_accept_filtered(
            _ptr(target_logits), _ptr(draft_logits), _ptr(draft_row), _ptr(tokens), _ptr(parent),
            B, n, V, R, D, float(temperature), int(seed) & (2**64 - 1), int(top_k), float(top_p),
            _ptr(accept_len), _ptr(path), _ptr(emit), _ptr(row_stats), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(_status(dev_status, dev)),
            _stream(stream)))
        return accept_len, path, emit
    if t2d is not None:
        _dev(t2d, "t2d", torch.int32)
        _check("eagle_verify_accept_d2t", lib().eagle_verify_accept_d2t(
            _ptr(target_logits), _ptr(draft_logits), _ptr(draft_row), _ptr(tokens), _ptr(parent),
            B, n, V, R, Vd, _ptr(t2d), D, float(temperature), int(seed) & (2**64 - 1),
            _ptr(accept_len), _ptr(path), _ptr(emit), _ptr(row_stats),
            _ptr(_status(dev_status, dev)), _stream(stream)))
        return accept_len, path, emit
    if draft_logits is not None and Vd != V:
        raise ValueError("draft rows over another vocabulary need t2d")
    _check("eagle_verify_accept", lib().eagle_verify_accept(
        _ptr(target_logits), _ptr(draft_logits), _ptr(draft_row), _ptr(tokens), _ptr(parent),
        B, n, V, R, D, float(temperature), int(seed) & (2**64 - 1),
        _ptr(accept_len), _ptr(path), _ptr(emit), _ptr(row_stats),
        _ptr(_status(dev_status, dev)), _stream(stream)))
    return accept_len, path, emit


def eagle_verify_accept_sharded(target_shards, draft_shards, shard_begin, tokens, parent, max_depth,
                                temperature, seed, draft_row=None, accept_len=None, path=None,
                                emit=None, row_stats=None, dev_status=None, stream=None):
    """Vocab-parallel verify: shard r of every target row ([B, n, Vr]) and draft row
    ([B, R, Vr]) holds the ids shard_begin[r] .. shard_begin[r+1]-1 (shard_begin: S + 1
    ints, 0 first, V last).  Returns (accept_len, path, emit) as eagle_verify_accept."""
    S = len(target_shards)
    begin = [int(x) for x in shard_begin]
    if len(begin) != S + 1:
        raise ValueError("shard_begin needs one entry per shard plus the vocabulary size")
    for r, t in enumerate(target_shards):
        _dev(t, f"target_shards[{r}]", torch.float32)
        if t.shape[-1] != begin[r + 1] - begin[r]:
            raise ValueError(f"target_shards[{r}] does not hold ids {begin[r]}..{begin[r + 1] - 1}")
    B, n = target_shards[0].shape[:2]
    V = begin[-1]
    R = n
    dptrs = None
    if draft_shards is not None:
        if len(draft_shards) != S:
            raise ValueError("one draft shard per target shard")
        for r, t in enumerate(draft_shards):
            _dev(t, f"draft_shards[{r}]", torch.float32)
        R = draft_shards[0].shape[1]
        dptrs = (ctypes.c_void_p * S)(*[t.data_ptr() for t in draft_shards])
    tptrs = (ctypes.c_void_p * S)(*[t.data_ptr() for t in target_shards])
    cbeg = (ctypes.c_int32 * (S + 1))(*begin)
    _dev(tokens, "tokens", torch.int32)
    _dev(parent, "parent", torch.int32)
    if draft_row is not None:
        _dev(draft_row, "draft_row", torch.int32)
    dev = tokens.device
    D = int(max_depth)
    accept_len = _empty(B, torch.int32, dev, stream) if accept_len is None else accept_len
    path = _empty((B, D + 1), torch.int32, dev, stream) if path is None else path
    emit = _empty((B, D + 1), torch.int32, dev, stream) if emit is None else emit
    if row_stats is not None:
        _dev(row_stats, "row_stats", torch.float32)
    _check("eagle_verify_accept_sharded", lib().eagle_verify_accept_sharded(
        tptrs, dptrs, cbeg, S, _ptr(draft_row), _ptr(tokens), _ptr(parent), B, n, V, R, D,
        float(temperature), int(seed) & (2**64 - 1), _ptr(accept_len), _ptr(path), _ptr(emit),
        _ptr(row_stats), _ptr(_status(dev_status, dev)), _stream(stream)))
    return accept_len, path, emit


def eagle_kv_compact(k_cache, v_cache, kv_len, path, accept_len, max_depth, dev_status=None,
                     stream=None):
    """k/v cache [n_layers,B,Hkv,Lmax,d] bf16 (in place); kv_len updated in place."""
    _dev(k_cache, "k_cache", torch.bfloat16)
    _dev(v_cache, "v_cache", torch.bfloat16)
    _dev(kv_len, "kv_len", torch.int32)
    _dev(path, "path", torch.int32)
    _dev(accept_len, "accept_len", torch.int32)
    nl, B, Hkv, Lmax, d = k_cache.shape
    _check("eagle_kv_compact", lib().eagle_kv_compact(
        _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(path), _ptr(accept_len),
        nl, B, Hkv, d, Lmax, int(max_depth), _ptr(_status(dev_status, k_cache.device)),
        _stream(stream)))


# ---------------------------------------------------------------- prompts and the 8-bit cache
KV8_BLOCK = 32      # cache rows that share a scale (EAGLE_KV8_BLOCK)


def _args(fn, dev, specs):
    """Checks (tensor, name, dtype, shape) rows: dense CUDA tensors on device `dev`.  These calls
    take microseconds on the GPU, so the checks are one pass of cheap tests; what is wrong
    is worked out only when something is."""
    for t, name, dtype, shape in specs:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a CUDA tensor")
        if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
                or not t.is_contiguous()):
            _dev(t, name, dtype)
            if t.shape != shape:
                raise ValueError(f"{fn}: {name} must be {list(shape)}, got {list(t.shape)}")
            raise ValueError(f"{fn}: {name} is on {t.device}, other tensors on cuda:{dev}")


def _token_rows(fn, t, name):
    """bf16 [T, H, d] rows whose tokens may be strided (a slice of a fused projection's
    output); returns the token stride in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{fn}: {name} must be [T, H, d]")
    T, H, d = t.shape
    if t.is_contiguous():
        return H * d
    s0, s1, s2 = t.stride()
    if not ((d == 1 or s2 == 1) and (H == 1 or s1 == d)):
        raise ValueError(f"{fn}: {name}'s heads must be dense within a token")
    if T > 1 and (s0 < H * d or s0 % 8 != 0):
        raise ValueError(f"{fn}: {name}'s token stride must be a multiple of 8, at least H * d")
    return s0 if T > 1 else H * d


def _launch(fn, dev, stream, args):
    """Calls the library on device `dev`, on `stream` or that device's current one."""
    f = getattr(lib(), fn)
    if torch._C._cuda_getDevice() == dev:
        raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
        code = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            code = f(*args, _stream(stream))
    if code != 0:
        raise EagleError(fn, code)


def _status_ptr(fn, dev, dev_status):
    if dev_status is None:
        return None
    _dev(dev_status, "dev_status", torch.int32)
    if dev_status.get_device() != dev:
        raise ValueError(f"{fn}: dev_status is on {dev_status.device}, other tensors on cuda:{dev}")
    return dev_status.data_ptr()


def kv8_cache(n_layers, B, Hkv, Lmax, d=128, device="cuda"):
    """An empty 8-bit cache: (k8, v8, k_scale, v_scale) for the calls below, codes
    [n_layers, B, Hkv, Lmax, d] and scales [n_layers, B, Hkv, ceil(Lmax / KV8_BLOCK)]."""
    codes = [torch.zeros(n_layers, B, Hkv, Lmax, d, dtype=torch.uint8, device=device)
             .view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones(n_layers, B, Hkv, -(-Lmax // KV8_BLOCK), device=device) for _ in range(2)]
    return (*codes, *scales)


def _kv8_specs(k8, v8, k_scale, v_scale, lead, Lmax, d):
    code, scale = (*lead, Lmax, d), (*lead, -(-Lmax // KV8_BLOCK))
    return ((k8, "k8", torch.float8_e4m3fn, code), (v8, "v8", torch.float8_e4m3fn, code),
            (k_scale, "k_scale", torch.float32, scale), (v_scale, "v_scale", torch.float32, scale))


def _cache_rows(fn, k8):
    if not isinstance(k8, torch.Tensor) or k8.dim() < 2:
        raise TypeError("k8 must be a CUDA tensor")
    return k8.shape[-2]


def eagle_prompt_attn(q, k, v, cu_q, cu_k=None, scale=None, out=None, lse=None, return_lse=False,
                      dev_status=None, stream=None):
    """Causal attention of packed prompts.  q [Tq,Hq,d], k / v [Tk,Hkv,d] bf16 (tokens may
    be strided), cu_q / cu_k int32 [B+1] (cu_k None: cu_q).  The queries of a sequence are
    the last positions of its keys.  Returns out [Tq,Hq,d], or (out, lse [Tq,Hq] f32)
    with return_lse or an lse tensor."""
    fn = "eagle_prompt_attn"
    sq, sk, sv = _token_rows(fn, q, "q"), _token_rows(fn, k, "k"), _token_rows(fn, v, "v")
    cu_k = cu_q if cu_k is None else cu_k
    Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[:2]
    if k.shape != (Tk, Hkv, d) or v.shape != k.shape:
        raise ValueError(f"{fn}: k and v must be [Tk, Hkv, {d}]")
    dev = q.get_device()
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"{fn}: q, k and v are on different devices")
    _dev(cu_q, "cu_q", torch.int32)
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError(f"{fn}: cu_q must be [B + 1]")
    B = cu_q.shape[0] - 1
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _empty((Tq, Hq, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((Tq, Hq), torch.float32, q.device, stream)
    _args(fn, dev, ((cu_q, "cu_q", torch.int32, cu_q.shape), (cu_k, "cu_k", torch.int32, cu_q.shape),
                    (out, "out", torch.bfloat16, q.shape)))
    if lse is not None:
        _args(fn, dev, ((lse, "lse", torch.float32, (Tq, Hq)),))
    _launch(fn, dev, stream, (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), out.data_ptr(),
        _ptr(lse), Tq, Tk, B, Hq, Hkv, d, sq, sk, sv, scale, _status_ptr(fn, dev, dev_status)))
    return out if lse is None else (out, lse)


def eagle_kv8_append(k, v, cu, pos, k8, v8, k_scale, v_scale, dev_status=None, stream=None):
    """Quantises one layer's new rows k / v [T,Hkv,d] bf16 (tokens may be strided; sequence
    b has rows cu[b] .. cu[b+1]-1) into the cache at rows pos[b] on, in place."""
    fn = "eagle_kv8_append"
    sk, sv = _token_rows(fn, k, "k"), _token_rows(fn, v, "v")
    T, Hkv, d = k.shape
    if v.shape != k.shape:
        raise ValueError(f"{fn}: v must be {list(k.shape)}, got {list(v.shape)}")
    _dev(pos, "pos", torch.int32)
    B, Lmax, dev = pos.numel(), _cache_rows(fn, k8), k.get_device()
    if v.get_device() != dev:
        raise ValueError(f"{fn}: k and v are on different devices")
    _args(fn, dev, ((pos, "pos", torch.int32, (B,)), (cu, "cu", torch.int32, (B + 1,)),
                    *_kv8_specs(k8, v8, k_scale, v_scale, (B, Hkv), Lmax, d)))
    _launch(fn, dev, stream, (
        k.data_ptr(), v.data_ptr(), cu.data_ptr(), pos.data_ptr(), k8.data_ptr(), v8.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), T, B, Hkv, d, Lmax, sk, sv,
        _status_ptr(fn, dev, dev_status)))


def eagle_kv8_commit(k_tree, v_tree, k8, v8, k_scale, v_scale, kv_len, path, accept_len, max_depth,
                     kv_len_out=None, dev_status=None, stream=None):
    """Quantises the accepted path's rows of the tree's K / V [n_layers,B,n,Hkv,d] bf16
    into the cache behind kv_len; kv_len is advanced in place, or into kv_len_out."""
    fn = "eagle_kv8_commit"
    _dev(k_tree, "k_tree", torch.bfloat16)
    if k_tree.dim() != 5:
        raise ValueError(f"{fn}: k_tree must be [n_layers, B, n, Hkv, d]")
    kv_len_out = kv_len if kv_len_out is None else kv_len_out
    nl, B, n, Hkv, d = k_tree.shape
    D, Lmax, dev = int(max_depth), _cache_rows(fn, k8), k_tree.get_device()
    i32 = torch.int32
    _args(fn, dev, ((v_tree, "v_tree", torch.bfloat16, k_tree.shape),
                    *_kv8_specs(k8, v8, k_scale, v_scale, (nl, B, Hkv), Lmax, d),
                    (kv_len, "kv_len", i32, (B,)), (kv_len_out, "kv_len_out", i32, (B,)),
                    (path, "path", i32, (B, D + 1)), (accept_len, "accept_len", i32, (B,))))
    _launch(fn, dev, stream, (
        k_tree.data_ptr(), v_tree.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), kv_len.data_ptr(), kv_len_out.data_ptr(), path.data_ptr(),
        accept_len.data_ptr(), nl, B, n, Hkv, d, Lmax, D, _status_ptr(fn, dev, dev_status)))
    return kv_len_out


@functools.lru_cache(maxsize=256)
def _tree_attn_kv8_workspace_size(dev, B, n, Hq, Hkv, head_dim, Lmax) -> int:
    with torch.cuda.device(dev):
        return int(lib().eagle_tree_attn_kv8_workspace_size(B, n, Hq, Hkv, head_dim, Lmax))


def tree_attn_kv8_workspace_size(B, n, Hq, Hkv, head_dim, Lmax) -> int:
    return int(lib().eagle_tree_attn_kv8_workspace_size(B, n, Hq, Hkv, head_dim, Lmax))


def eagle_tree_attn_kv8(q, k8, v8, k_scale, v_scale, k_tree, v_tree, kv_len, parent, scale=None,
                        out=None, workspace=None, dev_status=None, stream=None):
    """Tree attention over the 8-bit cache of one layer.  q [B,n,Hq,d] bf16, the cache
    [B,Hkv,Lmax,d], k_tree / v_tree [B,n,Hkv,d] bf16 (the tree's own rows), kv_len [B],
    parent [B,n] int32.  n = 1 with parent -1 is ordinary decoding."""
    fn = "eagle_tree_attn_kv8"
    _dev(q, "q", torch.bfloat16)
    _dev(k_tree, "k_tree", torch.bfloat16)
    if q.dim() != 4 or k_tree.dim() != 4:
        raise ValueError(f"{fn}: q must be [B, n, Hq, d] and k_tree [B, n, Hkv, d]")
    B, n, Hq, d = q.shape
    Hkv, Lmax, dev = k_tree.shape[2], _cache_rows(fn, k8), q.get_device()
    bf16, tree = torch.bfloat16, (B, n, Hkv, d)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _args(fn, dev, (*_kv8_specs(k8, v8, k_scale, v_scale, (B, Hkv), Lmax, d),
                    (k_tree, "k_tree", bf16, tree), (v_tree, "v_tree", bf16, tree),
                    (kv_len, "kv_len", torch.int32, (B,)), (parent, "parent", torch.int32, (B, n)),
                    (out, "out", bf16, q.shape)))
    ws_bytes = 0
    if workspace is None:
        ws_bytes = _tree_attn_kv8_workspace_size(dev, B, n, Hq, Hkv, d, Lmax)
        if ws_bytes:
            workspace = _empty(ws_bytes, torch.uint8, q.device, stream)
    else:
        _dev(workspace, "workspace")
        if workspace.get_device() != dev:
            raise ValueError(f"{fn}: workspace is on {workspace.device}, other tensors on cuda:{dev}")
        ws_bytes = workspace.numel() * workspace.element_size()
    _launch(fn, dev, stream, (
        q.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        k_tree.data_ptr(), v_tree.data_ptr(), kv_len.data_ptr(), parent.data_ptr(), out.data_ptr(),
        B, n, Hq, Hkv, d, Lmax, scale, _ptr(workspace), ws_bytes,
        _status_ptr(fn, dev, dev_status)))
    return out


# ---------------------------------------------------------------- the paged cache
def paged_cache(n_layers, n_pages, Hkv, page, B, max_pages, d=128, device="cuda"):
    """An empty paged cache: (k_pages, v_pages, page_table, held, refs) for the calls below, pages
    [n_layers, n_pages, Hkv, page, d] and, for B sequences, a table [B, max_pages]."""
    pages = [torch.zeros(n_layers, n_pages, Hkv, page, d, dtype=torch.bfloat16, device=device)
             for _ in range(2)]
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=device)
    return (*pages, table, *(torch.zeros(m, dtype=torch.int32, device=device) for m in (B, n_pages)))


def _dims(fn, t, name, n, what):
    """The shape of a tensor of n dimensions."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != n:
        raise ValueError(f"{fn}: {name} must be {what}")
    return t.shape


_PAGES, _LAYER = "[n_layers, N, Hkv, page, d]", "[N, Hkv, page, d]"


def _launch_with_workspace(fn, dev, stream, workspace, need, head, tail):
    """_launch with (workspace, its bytes) between the arguments of head and tail: the caller's, or
    `need` bytes of the stream's pool.  Those go back to it as soon as the call is enqueued, for
    work behind it on that stream: half the time of a tensor, in calls of a few microseconds."""
    if workspace is not None:
        _dev(workspace, "workspace")
        if workspace.get_device() != dev:
            raise ValueError(f"{fn}: workspace is on {workspace.device}, other tensors on cuda:{dev}")
        size = workspace.numel() * workspace.element_size()
        return _launch(fn, dev, stream, (*head, workspace.data_ptr(), size, *tail))
    if not need:
        return _launch(fn, dev, stream, (*head, None, 0, *tail))
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _launch_with_workspace(fn, dev, stream, None, need, head, tail)
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, raw)
    try:
        _launch(fn, dev, stream, (*head, ptr, need, *tail))
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(ptr)


@functools.lru_cache(maxsize=256)
def _pages_workspace_size(B, N, P) -> int:
    return pages_workspace_size(B, N, P)


def pages_workspace_size(B, N, P) -> int:
    return int(lib().eagle_pages_workspace_size(B, N, P))


def eagle_pages_assign(k_pages, v_pages, page_table, held, refs, kv_len, grow, src=None,
                       workspace=None, dev_status=None, stream=None):
    """Room for grow [B] rows behind each sequence's kv_len [B], after slot b went on with what
    slot src[b] held (None: its own; -1: nothing).  page_table [B,P], held [B], refs [N] and kv_len
    (int32) are updated in place; rows of pages that are shared no longer are copied in every
    layer of k_pages / v_pages [n_layers,N,Hkv,page,d] bf16.  All or nothing: a refused call sets
    dev_status and leaves the old table, with which the calls behind it go on (see eagle.h)."""
    fn = "eagle_pages_assign"
    nl, N, Hkv, page, d = shape = _dims(fn, k_pages, "k_pages", 5, _PAGES)
    B, P = table = _dims(fn, page_table, "page_table", 2, "[B, P]")
    dev, i32, bf16 = k_pages.get_device(), torch.int32, torch.bfloat16
    specs = ((k_pages, "k_pages", bf16, shape), (v_pages, "v_pages", bf16, shape),
             (page_table, "page_table", i32, table), (held, "held", i32, (B,)), (refs, "refs", i32, (N,)),
             (kv_len, "kv_len", i32, (B,)), (grow, "grow", i32, (B,)))
    _args(fn, dev, specs if src is None else (*specs, (src, "src", i32, (B,))))
    _launch_with_workspace(fn, dev, stream, workspace, _pages_workspace_size(B, N, P), (
        k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), held.data_ptr(), refs.data_ptr(),
        kv_len.data_ptr(), grow.data_ptr(), _ptr(src), nl, B, N, Hkv, page, d, P),
        (_status_ptr(fn, dev, dev_status),))


def eagle_pages_commit(k_pages, v_pages, page_table, kv_len, path, accept_len, max_depth,
                       kv_len_out=None, dev_status=None, stream=None):
    """Moves the accepted path's rows behind the committed ones in every layer of the pages
    [n_layers,N,Hkv,page,d] bf16; kv_len is advanced in place, or into kv_len_out."""
    fn = "eagle_pages_commit"
    nl, N, Hkv, page, d = _dims(fn, k_pages, "k_pages", 5, _PAGES)
    B, P = _dims(fn, page_table, "page_table", 2, "[B, P]")
    kv_len_out = kv_len if kv_len_out is None else kv_len_out
    D, dev, i32, bf16 = int(max_depth), k_pages.get_device(), torch.int32, torch.bfloat16
    _args(fn, dev, ((k_pages, "k_pages", bf16, k_pages.shape), (v_pages, "v_pages", bf16, k_pages.shape),
                    (page_table, "page_table", i32, (B, P)), (kv_len, "kv_len", i32, (B,)),
                    (kv_len_out, "kv_len_out", i32, (B,)), (path, "path", i32, (B, D + 1)),
                    (accept_len, "accept_len", i32, (B,))))
    _launch(fn, dev, stream, (
        k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(),
        kv_len_out.data_ptr(), path.data_ptr(), accept_len.data_ptr(), nl, B, N, Hkv, page, d, P, D,
        _status_ptr(fn, dev, dev_status)))
    return kv_len_out


def eagle_qkv_rope(q, k, v, inv_freq, pos, cu=None, parent=None, q_weight=None, k_weight=None,
                   eps=1e-6, interleaved=False, k_pages=None, v_pages=None, page_table=None,
                   q_out=None, k_out=None, dev_status=None, stream=None):
    """Norms of q's and k's heads (where weights [d] bf16 are given) and their rotation by
    position, and k and v into the cache's pages (one layer, [N,Hkv,page,d] bf16) where those are
    given.  q [T,Hq,d], k / v [T,Hkv,d] bf16 (tokens may be strided), inv_freq f32
    [rot_dim / 2], pos int32 [B]: the rows that each sequence holds.  The tokens are packed by cu
    [B+1], or the nodes of trees with parent [B,n] (T = B * n).  Returns (q_out [T,Hq,d], k_out
    [T,Hkv,d]); with pages, k_out is written only if it is given."""
    fn = "eagle_qkv_rope"
    sq, sk = _token_rows(fn, q, "q"), _token_rows(fn, k, "k")
    T, Hq, d = q.shape
    Hkv, dev, i32, bf16 = k.shape[1], q.get_device(), torch.int32, torch.bfloat16
    if k.shape != (T, Hkv, d):
        raise ValueError(f"{fn}: k must be [{T}, Hkv, {d}], got {list(k.shape)}")
    if (cu is None) == (parent is None):
        raise ValueError(f"{fn}: either cu or parent")
    _dev(pos, "pos", i32)
    _dev(inv_freq, "inv_freq", torch.float32)
    B, n = pos.numel(), 0
    if parent is not None:
        _dev(parent, "parent", i32)
        n = T // B if B else parent.shape[1] if parent.dim() == 2 else 0
    specs = [(pos, "pos", i32, (B,)), (inv_freq, "inv_freq", torch.float32, (inv_freq.numel(),)),
             (cu, "cu", i32, (B + 1,)) if parent is None else (parent, "parent", i32, (B, n))]
    N = page = P = sv = 0
    pages = k_pages is not None or v_pages is not None or page_table is not None
    if pages:
        N, _, page, _ = _dims(fn, k_pages, "k_pages", 4, _LAYER)
        P = _dims(fn, page_table, "page_table", 2, "[B, P]")[1]
        sv = _token_rows(fn, v, "v")
        if v.shape != k.shape or v.get_device() != dev:
            raise ValueError(f"{fn}: v must be like k")
        specs += [(k_pages, "k_pages", bf16, (N, Hkv, page, d)), (v_pages, "v_pages", bf16, (N, Hkv, page, d)),
                  (page_table, "page_table", i32, (B, P))]
    elif k_out is None:
        k_out = _empty((T, Hkv, d), bf16, q.device, stream)
    if k.get_device() != dev:
        raise ValueError(f"{fn}: q and k are on different devices")
    if q_out is None:
        q_out = _empty((T, Hq, d), bf16, q.device, stream)
    specs.append((q_out, "q_out", bf16, (T, Hq, d)))
    if k_out is not None:
        specs.append((k_out, "k_out", bf16, (T, Hkv, d)))
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            specs.append((w, name, bf16, (d,)))
    _args(fn, dev, specs)
    _launch(fn, dev, stream, (
        q.data_ptr(), k.data_ptr(), v.data_ptr() if pages else None, _ptr(q_weight), _ptr(k_weight),
        inv_freq.data_ptr(), _ptr(cu), _ptr(parent), pos.data_ptr(), q_out.data_ptr(), _ptr(k_out),
        _ptr(k_pages), _ptr(v_pages), _ptr(page_table), T, B, n, Hq, Hkv, d, 2 * inv_freq.numel(),
        bool(interleaved), eps, sq, sk, sv, N, page, P, _status_ptr(fn, dev, dev_status)))
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def _tree_attn_paged_workspace_size(dev, B, n, Hq, Hkv, head_dim, page, P) -> int:
    with torch.cuda.device(dev):
        return tree_attn_paged_workspace_size(B, n, Hq, Hkv, head_dim, page, P)


def tree_attn_paged_workspace_size(B, n, Hq, Hkv, head_dim, page, P) -> int:
    return int(lib().eagle_tree_attn_paged_workspace_size(B, n, Hq, Hkv, head_dim, page, P))


def eagle_tree_attn_paged(q, k_pages, v_pages, page_table, kv_len, parent, scale=None, out=None,
                          workspace=None, dev_status=None, stream=None):
    """Tree attention over the pages of one layer [N,Hkv,page,d] bf16, the tree's rows in them
    behind kv_len.  q [B,n,Hq,d] bf16, page_table [B,P], kv_len [B], parent [B,n] int32.  n = 1 with
    parent -1 is ordinary decoding."""
    fn = "eagle_tree_attn_paged"
    _dev(q, "q", torch.bfloat16)
    if q.dim() != 4:
        raise ValueError(f"{fn}: q must be [B, n, Hq, d]")
    B, n, Hq, d = q.shape
    N, Hkv, page, _ = _dims(fn, k_pages, "k_pages", 4, _LAYER)
    P, dev = _dims(fn, page_table, "page_table", 2, "[B, P]")[1], q.get_device()
    bf16, i32 = torch.bfloat16, torch.int32
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _empty_like(q, stream)
    _args(fn, dev, ((k_pages, "k_pages", bf16, (N, Hkv, page, d)), (v_pages, "v_pages", bf16, (N, Hkv, page, d)),
                    (page_table, "page_table", i32, (B, P)), (kv_len, "kv_len", i32, (B,)),
                    (parent, "parent", i32, (B, n)), (out, "out", bf16, q.shape)))
    _launch_with_workspace(fn, dev, stream, workspace, _tree_attn_paged_workspace_size(dev, B, n, Hq, Hkv, d, page, P), (
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(),
        parent.data_ptr(), out.data_ptr(), B, n, Hq, Hkv, d, N, page, P, scale),
        (_status_ptr(fn, dev, dev_status),))
    return out


def expand_scratch_size(B, V, top_k) -> int:
    return int(lib().eagle2_expand_scratch_size(B, V, top_k))


def eagle2_expand(level, final, logits, top_k, depth, n_out, tree_state, hidden=None,
                  lm_head_w=None, out_tokens=None, out_parent=None, out_draft_row=None,
                  frontier_tokens=None, dev_status=None, stream=None, partials=None, d2t=None):
    """One EAGLE-2 level over draft-logit storage logits [B, R, V] (f32).  With a
    partials buffer the level's statistics come from the GEMM epilogue's per-tile
    partials (written by this call's GEMM when hidden is given, else by a prior
    eagle_lmhead_gemm(..., partials=...) for the level's rows) and its top-k from a
    rescan of the few tiles that can hold it.  With d2t (int32 [V]) V is a draft
    vocabulary and the tokens written are target ids d + d2t[d]."""
    _dev(logits, "logits", torch.float32)
    _dev(tree_state, "tree_state")
    B, R, V = logits.shape
    H = 0
    if hidden is not None:
        _dev(hidden, "hidden", torch.bfloat16)
        _dev(lm_head_w, "lm_head_w", torch.bfloat16)
        H = hidden.shape[-1]
    for name, t in (("out_tokens", out_tokens), ("out_parent", out_parent),
                    ("out_draft_row", out_draft_row), ("frontier_tokens", frontier_tokens)):
        if t is not None:
            _dev(t, name, torch.int32)
    nbytes = tree_state.numel() * tree_state.element_size()
    sbytes = 0
    if partials is not None:
        _dev(partials, "partials", torch.float32)
        sbytes = partials.numel() * partials.element_size()
    if d2t is not None:
        _dev(d2t, "d2t", torch.int32)
        if d2t.numel() != V:
            raise ValueError("d2t needs one entry per draft id")
        _check("eagle2_expand_d2t", lib().eagle2_expand_d2t(
            int(level), int(final), _ptr(hidden), _ptr(lm_head_w), _ptr(logits), B, H, V, top_k,
            depth, n_out, _ptr(tree_state), nbytes, _ptr(partials), sbytes, _ptr(d2t),
            _ptr(out_tokens), _ptr(out_parent), _ptr(out_draft_row), _ptr(frontier_tokens),
            _ptr(_status(dev_status, logits.device)), _stream(stream)))
        return
    _check("eagle2_expand", lib().eagle2_expand(
        int(level), int(final), _ptr(hidden), _ptr(lm_head_w), _ptr(logits), B, H, V, top_k, depth,
        n_out, _ptr(tree_state), nbytes, _ptr(partials), sbytes, _ptr(out_tokens), _ptr(out_parent),
        _ptr(out_draft_row), _ptr(frontier_tokens), _ptr(_status(dev_status, logits.device)),
        _stream(stream)))


def eagle2_tree_candidates(tree_state, B, top_k, depth, stream=None):
    """Every candidate of a tree state as CUDA tensors [B, C]: dict(value, conf (f32),
    token, parent, depth, draft_row (int32)), C = 1 + top_k + (depth - 1) * top_k^2."""
    _dev(tree_state, "tree_state")
    C = 1 + top_k + (depth - 1) * top_k * top_k
    dev = tree_state.device
    out = {name: _empty((B, C), torch.float32, dev, stream) for name in ("value", "conf")}
    for name in ("token", "parent", "depth", "draft_row"):
        out[name] = _empty((B, C), torch.int32, dev, stream)
    nbytes = tree_state.numel() * tree_state.element_size()
    _check("eagle2_tree_candidates", lib().eagle2_tree_candidates(
        _ptr(tree_state), nbytes, B, top_k, depth, _ptr(out["value"]), _ptr(out["conf"]),
        _ptr(out["token"]), _ptr(out["parent"]), _ptr(out["depth"]), _ptr(out["draft_row"]),
        _stream(stream)))
    return out


def eagle_static_tree(choices):
    """Plan a static draft tree from its choices (rank paths from the root) on the host.
    Returns dict(parent, rank, depth, draft_row) of int32 numpy arrays [n]."""
    import numpy as np
    n_choices = len(choices)
    max_len = max((len(c) for c in choices), default=1)
    ranks = np.zeros((max(n_choices, 1), max_len), np.int32)
    lens = np.zeros(max(n_choices, 1), np.int32)
    for i, c in enumerate(choices):
        ranks[i, :len(c)] = c
        lens[i] = len(c)
    n_max = n_choices + 1
    out = {k: np.zeros(n_max, np.int32) for k in ("parent", "rank", "depth", "draft_row")}
    n_nodes = np.zeros(1, np.int32)
    adr = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    _check("eagle_static_tree", lib().eagle_static_tree(
        adr(ranks), adr(lens), n_choices, max_len, n_max, adr(out["parent"]), adr(out["rank"]),
        adr(out["depth"]), adr(out["draft_row"]), adr(n_nodes)))
    n = int(n_nodes[0])
    return {k: v[:n] for k, v in out.items()}


def eagle_static_tree_level(level, logits, parent, rank, depth, draft_row, tokens,
                            dev_status=None, stream=None):
    """Tokens of the nodes at depth `level` of a static tree (device int32 arrays [n]),
    from the internal nodes' draft rows logits [B, R, V] (f32), into tokens [B, n]."""
    _dev(logits, "logits", torch.float32)
    for name, t in (("parent", parent), ("rank", rank), ("depth", depth),
                    ("draft_row", draft_row), ("tokens", tokens)):
        _dev(t, name, torch.int32)
    B, R, V = logits.shape
    _check("eagle_static_tree_level", lib().eagle_static_tree_level(
        int(level), _ptr(logits), _ptr(parent), _ptr(rank), _ptr(depth), _ptr(draft_row),
        parent.numel(), B, R, V, _ptr(tokens), _ptr(_status(dev_status, logits.device)),
        _stream(stream)))


def eagle2_expand_static_state(level, final, logits, top_k, depth, n_out, hidden=None,
                               lm_head_w=None, out_tokens=None, out_parent=None,
                               out_draft_row=None, frontier_tokens=None, dev_status=None,
                               stream=None):
    """eagle2_expand with the tree state kept in the library's own fixed device array
    (no scratch argument; one tree at a time per device, levels in order)."""
    _dev(logits, "logits", torch.float32)
    B, R, V = logits.shape
    H = 0
    if hidden is not None:
        _dev(hidden, "hidden", torch.bfloat16)
        _dev(lm_head_w, "lm_head_w", torch.bfloat16)
        H = hidden.shape[-1]
    for name, t in (("out_tokens", out_tokens), ("out_parent", out_parent),
                    ("out_draft_row", out_draft_row), ("frontier_tokens", frontier_tokens)):
        if t is not None:
            _dev(t, name, torch.int32)
    _check("eagle2_expand_static_state", lib().eagle2_expand_static_state(
        int(level), int(final), _ptr(hidden), _ptr(lm_head_w), _ptr(logits), B, H, V, top_k,
        depth, n_out, _ptr(out_tokens), _ptr(out_parent), _ptr(out_draft_row),
        _ptr(frontier_tokens), _ptr(_status(dev_status, logits.device)), _stream(stream)))


def eagle_softmax_stats(logits, temperature, row_max=None, row_sum=None, row_argmax=None,
                        dev_status=None, stream=None, argmax=True):
    """(row_max, row_sum, row_argmax) of softmax(logits / T) per row.  At T > 0 the
    argmax is computed only when `argmax` is true (or row_argmax is given); it is
    returned as None otherwise."""
    _dev(logits, "logits", torch.float32)
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    shp = logits.shape[:-1]
    if temperature > 0:
        row_max = _empty(shp, torch.float32, dev, stream) if row_max is None else row_max
        row_sum = _empty(shp, torch.float32, dev, stream) if row_sum is None else row_sum
    if row_argmax is None and (argmax or temperature <= 0):
        row_argmax = _empty(shp, torch.int32, dev, stream)
    _check("eagle_softmax_stats", lib().eagle_softmax_stats(
        _ptr(logits), rows, V, float(temperature), _ptr(row_max), _ptr(row_sum), _ptr(row_argmax),
        _ptr(_status(dev_status, dev)), _stream(stream)))
    return row_max, row_sum, row_argmax


def eagle_lmhead_gemm(hidden, w, out=None, ldo=None, rows_per_group=None, group_stride=0,
                      row_offset=0, dev_status=None, stream=None, partials=None):
    """out[row(m)] = hidden[m] . W^T, hidden [M,K], w [N,K] bf16, out f32.  With a
    partials buffer [M, ceil(N/256), 2] (f32) also each row's per-tile (max, sum of
    exponentials)."""
    _dev(hidden, "hidden", torch.bfloat16)
    _dev(w, "w", torch.bfloat16)
    M, K = hidden.shape
    N = w.shape[0]
    if out is None:
        out = _empty((M, N), torch.float32, hidden.device, stream)
    _dev(out, "out", torch.float32)
    ldo = N if ldo is None else ldo
    rpg = M if rows_per_group is None else rows_per_group
    if partials is not None:
        _dev(partials, "partials", torch.float32)
    _check("eagle_lmhead_gemm", lib().eagle_lmhead_gemm(
        _ptr(hidden), _ptr(w), _ptr(out), M, K, N, int(ldo), int(rpg), int(group_stride),
        int(row_offset), _ptr(partials), _ptr(_status(dev_status, hidden.device)),
        _stream(stream)))
    return out
