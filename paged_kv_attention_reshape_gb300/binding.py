"""Python binding of the C ABI: torch tensors in, data pointers and sizes out.

Argument marshalling only: every step of the computation runs in libpkv.so's CUDA kernels.
Tensors must be CUDA tensors on the current device; outputs that are not passed in are
allocated here with torch (the library itself never allocates). Calls are asynchronous on the
current torch stream unless ``stream`` is given; what a call on another stream is not given is
allocated there, so that nothing queued on the current stream still writes it.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib

CLASS_DECODE, CLASS_EXTEND, CLASS_PREFILL = _lib.CLASS_DECODE, _lib.CLASS_EXTEND, _lib.CLASS_PREFILL


class PkvError(RuntimeError):
    pass


def _check(status: int, what: str):
    if status != _lib.PKV_OK:
        raise PkvError(f"{what}: {_lib.STATUS.get(status, status)}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object around it (a few microseconds a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _other(stream) -> Optional[torch.cuda.Stream]:
    """The call's stream if it is another than the current one, else None."""
    if stream is None:
        return None
    handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if handle == (_stream(None).value or 0):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.default_stream() if handle in (0, 1) else torch.cuda.ExternalStream(handle)  # (1: the legacy default)


def _empty(shape, dtype, device, other) -> torch.Tensor:
    """A tensor that a call on `other` (None: the current stream) writes and the current stream reads. It comes from
    `other`'s memory: a block that the current stream has just given back may still be written by what is queued
    there, which the call does not wait for. Given back, it is kept until what the current stream has queued is done."""
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _scratch(need: int, workspace, device, other):
    """The caller's workspace if it is large enough, else one of `need` bytes (None for 0) from the memory of the
    call's stream, which is all that uses it."""
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        if not need:
            return workspace
        if other is None:
            return torch.empty(need, dtype=torch.uint8, device=device)
        with torch.cuda.stream(other):
            return torch.empty(need, dtype=torch.uint8, device=device)
    return workspace


def _need(t: torch.Tensor, dtype, name: str, contiguous: bool = True):
    if not t.is_cuda:
        raise PkvError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise PkvError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise PkvError(f"{name} must be contiguous")


_FP8 = (torch.uint8, torch.float8_e4m3fn)


def _is_number(scale, shape) -> bool:
    """Whether a scale is one for the whole tensor: a number, or a tensor of one element that is not a table."""
    return not isinstance(scale, torch.Tensor) or (scale.numel() == 1 and scale.shape != shape)


def _block_scales(k_scale, v_scale, nb: int, hkv: int, device_index: int):
    """Checks scale tensors [num_blocks, Hkv]; returns their addresses."""
    want = (nb, hkv)
    if (isinstance(k_scale, torch.Tensor) and isinstance(v_scale, torch.Tensor) and k_scale.dtype is torch.float32
            and v_scale.dtype is torch.float32 and k_scale.shape == want and v_scale.shape == want
            and k_scale.get_device() == device_index == v_scale.get_device() and k_scale.is_contiguous()
            and v_scale.is_contiguous()):
        return k_scale.data_ptr(), v_scale.data_ptr()
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if not isinstance(t, torch.Tensor):
            raise PkvError("k_scale and v_scale must both be numbers or both be tensors")
        _need(t, torch.float32, n)
        if tuple(t.shape) != (nb, hkv):
            raise PkvError(f"{n} must be [num_blocks, Hkv] = [{nb}, {hkv}], got {list(t.shape)}")
        if t.get_device() != device_index:
            raise PkvError(f"{n} must be on the cache's device")
    return k_scale.data_ptr(), v_scale.data_ptr()


def make_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale=1.0, v_scale=1.0) -> "_lib.PkvCache":
    """Describe one layer's paged cache: k_cache / v_cache [num_blocks, block_size, Hkv, D]
    with contiguous blocks (any stride between blocks). bf16 tensors are a bf16 cache; uint8
    or float8_e4m3fn tensors are an FP8 (E4M3) cache whose codes stand for e4m3(code) * scale.
    k_scale and v_scale are numbers (one scale for the tensor; a tensor of one element counts as one, and is
    read on the host) or fp32 tensors [num_blocks, Hkv] (a scale for each block and KV head)."""
    dtype = k_cache.dtype
    fp8 = dtype in _FP8
    shape = k_cache.shape
    nb, bs, hkv, d = shape
    st = k_cache.stride()
    stride = st[0]
    if not (k_cache.is_cuda and v_cache.is_cuda and (fp8 or dtype is torch.bfloat16) and v_cache.dtype is dtype
            and v_cache.shape == shape and v_cache.stride() == st and st[1] == hkv * d and st[2] == d and st[3] == 1):
        want = dtype if fp8 else torch.bfloat16
        for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, want, n, contiguous=False)
            if t.stride()[1:] != (hkv * d, d, 1):
                raise PkvError(f"{n}: each block must be contiguous [block_size, Hkv, D]")
        if k_cache.shape != v_cache.shape or stride != v_cache.stride(0):
            raise PkvError("k_cache and v_cache must have the same shape and block stride")
    if not (_is_number(k_scale, (nb, hkv)) and _is_number(v_scale, (nb, hkv))):
        if not fp8:
            raise PkvError("block scales belong to an FP8 cache")
        ks, vs = _block_scales(k_scale, v_scale, nb, hkv, k_cache.get_device())
        return _lib.PkvCache(k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, hkv, d, stride,
                             _lib.KV_FP8_E4M3_BLOCK, 1.0, 1.0, ks, vs)
    return _lib.PkvCache(k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, hkv, d, stride,
                         _lib.KV_FP8_E4M3 if fp8 else _lib.KV_BF16, float(k_scale), float(v_scale))


@dataclass
class Reqs:
    """A request set (pkv_reqs): order[bounds[cls]:bounds[cls+1]] when bounds is given, else
    order[:max_reqs] (or 0..max_reqs-1 without order). batch_reqs = R of the batch arrays."""
    max_reqs: int
    batch_reqs: int
    order: Optional[torch.Tensor] = None
    bounds: Optional[torch.Tensor] = None
    cls: int = 0

    def c(self) -> "_lib.PkvReqs":
        return _lib.PkvReqs(self.order.data_ptr() if self.order is not None else None,
                            self.bounds.data_ptr() if self.bounds is not None else None,
                            self.cls, self.max_reqs, self.batch_reqs)


def kv_cache_write(key, value, slot_mapping, k_cache, v_cache, stream=None, k_scale=1.0, v_scale=1.0):
    """Scatter key/value [T, Hkv, D] into the cache slots given by slot_mapping (int64 [T]);
    into an FP8 cache, quantised with the per-tensor scales."""
    lib = _lib.load()
    _need(key, torch.bfloat16, "key")
    _need(value, torch.bfloat16, "value")
    _need(slot_mapping, torch.int64, "slot_mapping")
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    _check(lib.pkv_kv_cache_write(_ptr(key), _ptr(value), _ptr(slot_mapping), slot_mapping.numel(),
                                  cache, _stream(stream)), "kv_cache_write")


def _token_rows(t: torch.Tensor, name: str, rows: int, heads: int, dim: int, device_index: int) -> int:
    """Checks bf16 rows [rows, heads, dim] whose tokens may lie apart (a slice of a fused projection);
    returns the elements between tokens."""
    if t.get_device() != device_index:  # -1 for a CPU tensor
        raise PkvError(f"{name} must be on the cache's device")
    if t.dtype is not torch.bfloat16:
        raise PkvError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (rows, heads, dim):
        raise PkvError(f"{name} must be [{rows}, {heads}, {dim}], got {list(t.shape)}")
    if t.is_contiguous():
        return heads * dim
    st = t.stride()
    if (dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim):
        raise PkvError(f"{name}: each token's heads must be contiguous")
    return st[0] if rows > 1 else heads * dim


def _token_index(t: torch.Tensor, name: str, rows: int, device_index: int) -> int:
    if t.get_device() != device_index or t.dtype is not torch.int64 or t.numel() != rows \
            or not t.is_contiguous():
        raise PkvError(f"{name} must be {rows} contiguous int64 entries on the cache's device")
    return t.data_ptr()


def _token_out(t: Optional[torch.Tensor], name: str, rows: int, heads: int, dim: int, like: torch.Tensor, other) -> torch.Tensor:
    if t is None:
        return _empty((rows, heads, dim), torch.bfloat16, like.device, other)
    if _token_rows(t, name, rows, heads, dim, like.get_device()) != heads * dim or not t.is_contiguous():
        raise PkvError(f"{name} must be contiguous")
    return t


def _head_norm(q_norm, k_norm, eps, dim: int, device_index: int) -> "_lib.PkvHeadNorm":
    some = k_norm if q_norm is None else q_norm
    for w, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if w is None:
            continue
        if w.get_device() != device_index or w.dtype not in (torch.bfloat16, torch.float32) or w.shape != (dim,) \
                or not w.is_contiguous() or w.dtype is not some.dtype:
            raise PkvError(f"{name} must be contiguous [{dim}] bf16 or fp32 on the cache's device, alike for q and k")
    return _lib.PkvHeadNorm(None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                            float(eps), 1 if some.dtype is torch.float32 else 0)


def kv_append(q, key, value, positions, slot_mapping, k_cache, v_cache, cos_sin=None, *, rope_offset=0,
              interleaved=False, q_out=None, k_out=None, k_scale=1.0, v_scale=1.0, stream=None, q_norm=None,
              k_norm=None, norm_eps=1e-6):
    """Rotate q and key by their positions and append key and value to the cache slots.

    q [T, Hq, D] (or None), key and value [T, Hkv, D] bf16, tokens any stride apart; positions and
    slot_mapping int64 [T] (slot < 0: a padding row, skipped); cos_sin fp32 [max_pos, n]: n/2 cosines
    then n/2 sines for dims rope_offset .. rope_offset + n - 1 of every head (None: no rotation). A
    bf16 or FP8 cache; with k_scale / v_scale tensors [num_blocks, Hkv] the scales of the blocks
    written are updated too. A latent cache: value and v_cache None. Returns (q_out, k_out): the
    rotated rows, [T, H, D] contiguous, allocated here when not given (rows of skipped tokens are
    left as they were).

    q_norm and k_norm, weights [D] (bf16 or fp32, both alike; either may be None): every query (key) head is
    divided by the root of its mean square plus norm_eps and multiplied by them before it is rotated
    (D a power of two of at most 512, no latent cache)."""
    lib = _lib.load()
    if (value is None) != (v_cache is None):
        raise PkvError("a latent cache has neither value nor v_cache; any other has both")
    cache = make_cache(k_cache, k_cache if v_cache is None else v_cache, k_scale, v_scale)
    dev, hkv, d = k_cache.get_device(), cache.num_kv_heads, cache.head_dim
    if dev != torch.cuda.current_device():
        raise PkvError("the cache must be on the current device")
    other = _other(stream)
    T = key.shape[0]
    k_stride = _token_rows(key, "key", T, hkv, d, dev)
    v_ptr, v_stride = None, 0
    if value is not None:
        v_ptr, v_stride = value.data_ptr(), _token_rows(value, "value", T, hkv, d, dev)
    hq, q_ptr, q_stride, qo_ptr = 0, None, 0, None
    if q is not None:
        hq = q.shape[1]
        q_ptr, q_stride = q.data_ptr(), _token_rows(q, "q", T, hq, d, dev)
        q_out = _token_out(q_out, "q_out", T, hq, d, k_cache, other)
        qo_ptr = q_out.data_ptr()
    k_out = _token_out(k_out, "k_out", T, hkv, d, k_cache, other)
    pos_ptr = None
    if cos_sin is not None:
        if cos_sin.get_device() != dev or cos_sin.dtype is not torch.float32 \
                or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise PkvError("cos_sin must be contiguous fp32 [max_pos, n] on the cache's device")
        rows, n = cos_sin.shape
        rope = _lib.PkvRope(cos_sin.data_ptr(), rows, n, int(rope_offset), 1 if interleaved else 0)
        pos_ptr = _token_index(positions, "positions", T, dev)
    else:
        rope = _lib.PkvRope(None, 0, 0, 0, 0)
    slots = _token_index(slot_mapping, "slot_mapping", T, dev)
    if q_norm is not None or k_norm is not None:
        norm = _head_norm(q_norm, k_norm, norm_eps, d, dev)
        _check(lib.pkv_kv_append_norm(q_ptr, q_stride, key.data_ptr(), k_stride, v_ptr, v_stride, pos_ptr, slots, T, hq,
                                      rope, norm, cache, qo_ptr, k_out.data_ptr(), _stream(stream)), "kv_append")
        return q_out, k_out
    _check(lib.pkv_kv_append(q_ptr, q_stride, key.data_ptr(), k_stride, v_ptr, v_stride, pos_ptr, slots, T, hq, rope,
                             cache, qo_ptr, k_out.data_ptr(), _stream(stream)), "kv_append")
    return q_out, k_out


def kv_block_pack(k_cache, v_cache, block_ids, dst=None, stream=None):
    """dst [2, n, block_size, Hkv, D] = (k_cache[block_ids], v_cache[block_ids])."""
    lib = _lib.load()
    _need(block_ids, torch.int32, "block_ids")
    cache = make_cache(k_cache, v_cache)
    n = block_ids.numel()
    if dst is None:
        dst = _empty((2, n) + tuple(k_cache.shape[1:]), k_cache.dtype, k_cache.device, _other(stream))
    _need(dst, k_cache.dtype, "dst")
    _check(lib.pkv_kv_block_pack(cache, _ptr(block_ids), n, _ptr(dst), _stream(stream)), "kv_block_pack")
    return dst


def kv_block_unpack(src, block_ids, k_cache, v_cache, stream=None):
    """k_cache[block_ids[i]] = src[0][i], v_cache[block_ids[i]] = src[1][i] (in place)."""
    lib = _lib.load()
    _need(src, k_cache.dtype, "src")
    _need(block_ids, torch.int32, "block_ids")
    cache = make_cache(k_cache, v_cache)
    n = block_ids.numel()
    if tuple(src.shape) != (2, n) + tuple(k_cache.shape[1:]):
        raise ValueError(f"src shape {tuple(src.shape)} does not match 2 x {n} blocks of {tuple(k_cache.shape[1:])}")
    _check(lib.pkv_kv_block_unpack(_ptr(src), _ptr(block_ids), n, cache, _stream(stream)), "kv_block_unpack")


class CacheLayers:
    """The layers of one pool of blocks, described once for kv_block_copy: k_caches and v_caches are lists of
    [num_blocks, block_size, Hkv, D] tensors alike in shape, stride and type (v_caches None: a latent cache);
    k_scales and v_scales, for a block-scaled cache, lists of fp32 [num_blocks, Hkv]. Scales that are numbers
    count for nothing here. The tensors are kept alive with the handle. Making one costs some 2 us a layer, so it is made
    once for a pool and kept."""

    def __init__(self, k_caches, v_caches=None, k_scales=None, v_scales=None):
        k_caches = list(k_caches)
        v_caches = k_caches if v_caches is None else list(v_caches)

        def per_layer(s, name):
            if s is None or not isinstance(s, (list, tuple)):
                return [1.0 if s is None else s] * len(k_caches)
            if len(s) != len(k_caches):
                raise PkvError(f"{name}: one for each layer")
            return list(s)

        k_scales, v_scales = per_layer(k_scales, "k_scales"), per_layer(v_scales, "v_scales")
        if not k_caches or len(v_caches) != len(k_caches):
            raise PkvError("k_caches and v_caches must hold one tensor for each layer")
        made = [make_cache(*layer) for layer in zip(k_caches, v_caches, k_scales, v_scales)]
        self.device_index = k_caches[0].get_device()
        if any(t.get_device() != self.device_index for t in k_caches + v_caches):
            raise PkvError("all layers must be on one device")
        self._layers = (_lib.PkvCache * len(made))(*made)
        self._kept = (k_caches, v_caches, k_scales, v_scales)

    def __len__(self):
        return len(self._layers)


def kv_block_copy(layers: CacheLayers, src_ids, dst_ids, stream=None):
    """In every layer, block dst_ids[i] becomes a copy of block src_ids[i] (int32 ids; a negative one skips the
    pair). A source may be copied many times; a destination must be in one pair only and be no pair's source."""
    lib = _lib.load()
    n, dev = src_ids.numel(), layers.device_index
    if dev != torch.cuda.current_device():
        raise PkvError("the cache must be on the current device")
    for t, name in ((src_ids, "src_ids"), (dst_ids, "dst_ids")):
        if t.dtype is not torch.int32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
            raise PkvError(f"{name} must be {n} contiguous int32 ids on the cache's device")
    _check(lib.pkv_kv_block_copy(layers._layers, len(layers._layers), src_ids.data_ptr(), dst_ids.data_ptr(), n,
                                 _stream(stream)), "kv_block_copy")


class LayerHandoff:
    """Per-layer handoff staging on a copy stream of its own (pkv_handoff_*): stage(slot, ...)
    packs one layer's blocks into dst after the work already on the compute stream, without
    holding up the compute stream; ready(slot, stream) orders a consumer after that pack;
    release(slot, stream) orders the slot's next stage after the consumer."""

    def __init__(self, num_slots: int, copy_stream: Optional[torch.cuda.Stream] = None):
        lib = _lib.load()
        self.copy_stream = copy_stream if copy_stream is not None else torch.cuda.Stream()
        self.num_slots = int(num_slots)
        h = ctypes.c_void_p()
        _check(lib.pkv_handoff_create(self.num_slots, _stream(self.copy_stream), ctypes.byref(h)), "handoff_create")
        self._h = h

    def stage(self, slot, k_cache, v_cache, block_ids, dst=None, compute_stream=None):
        lib = _lib.load()
        _need(block_ids, torch.int32, "block_ids")
        cache = make_cache(k_cache, v_cache)
        n = block_ids.numel()
        if dst is None:
            # allocated on the copy stream's behalf: the caching allocator must not hand it to
            # other work before the pack that writes it is done, nor to a later pack before the
            # current stream has read it
            dst = _empty((2, n) + tuple(k_cache.shape[1:]), k_cache.dtype, k_cache.device, self.copy_stream)
        _need(dst, k_cache.dtype, "dst")
        _check(lib.pkv_handoff_stage(self._h, int(slot), cache, _ptr(block_ids), n, _ptr(dst), _stream(compute_stream)),
               "handoff_stage")
        return dst

    def ready(self, slot, stream=None):
        _check(_lib.load().pkv_handoff_ready(self._h, int(slot), _stream(stream)), "handoff_ready")

    def release(self, slot, stream=None):
        _check(_lib.load().pkv_handoff_release(self._h, int(slot), _stream(stream)), "handoff_release")

    def close(self):
        if self._h is not None and self._h.value:
            _check(_lib.load().pkv_handoff_destroy(self._h), "handoff_destroy")
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def selftest_bounded_wait(limit_ns=10_000_000, stream=None):
    """Run a kernel whose barrier wait must run out after limit_ns (sets the TIMEOUT bit of the
    device error word; the context stays usable)."""
    _check(_lib.load().pkv_selftest_bounded_wait(int(limit_ns), _stream(stream)), "selftest_bounded_wait")


def batch_classify_reorder(cu_q, seq_lens, decode_threshold=1, perm=None, bounds=None,
                           cu_q_reordered=None, token_map=None, with_token_map=False,
                           num_tokens=None, stream=None):
    """Returns (perm, bounds[4], cu_q_reordered, token_map or None)."""
    lib = _lib.load()
    _need(cu_q, torch.int32, "cu_q")
    _need(seq_lens, torch.int32, "seq_lens")
    R = seq_lens.numel()
    dev, other = seq_lens.device, _other(stream)
    perm = perm if perm is not None else _empty(R, torch.int32, dev, other)
    bounds = bounds if bounds is not None else _empty(4, torch.int32, dev, other)
    cu_q_reordered = cu_q_reordered if cu_q_reordered is not None else _empty(R + 1, torch.int32, dev, other)
    if with_token_map and token_map is None:
        if num_tokens is None:
            raise PkvError("num_tokens (host) is needed for the token map")
        token_map = _empty(num_tokens, torch.int32, dev, other)
    T = token_map.numel() if token_map is not None else (num_tokens or 0)
    _check(lib.pkv_batch_classify_reorder(_ptr(cu_q), _ptr(seq_lens), R, decode_threshold, _ptr(perm),
                                          _ptr(bounds), _ptr(cu_q_reordered), _ptr(token_map), T,
                                          _stream(stream)), "batch_classify_reorder")
    return perm, bounds, cu_q_reordered, token_map


def _scale(scale, D):
    return float(scale) if scale is not None else 1.0 / math.sqrt(D)


def paged_decode_workspace_size(max_reqs, Hq, Hkv, D, max_seq_len) -> int:
    return int(_lib.load().pkv_paged_decode_workspace_size(max_reqs, Hq, Hkv, D, max_seq_len))


def _window(window, sinks):
    """The (window, sinks) of a windowed call as 32-bit integers (no row is further away than that; below zero they stay
    refused), or None for a call without a window."""
    if window is None:
        if sinks:
            raise PkvError("sinks belong to a window")
        return None
    return max(-1, min(int(window), 2**31 - 1)), max(-1, min(int(sinks), 2**31 - 1))


def _window_args(q, heads, dim, rows, reqs, index, out, lse, kv=(), workspace=None):
    """Checks the tensors of a windowed call: on the current device, as large as what the kernels read and write (q, the
    lengths, tables and new rows have passed _need). index: (tensor, name, least entries); kv: (tensor, name) rows
    of keys and values [rows, heads, dim]."""
    dev = q.get_device()
    if dev != torch.cuda.current_device():
        raise PkvError("q must be on the current device")
    n, hq, d = q.shape
    n *= hq
    if d != dim:
        raise PkvError(f"q must be [T, Hq, {dim}]")
    if reqs.order is not None or reqs.bounds is not None:
        index += ((reqs.order, "order", reqs.max_reqs if reqs.bounds is None else 0), (reqs.bounds, "bounds", reqs.cls + 2))
        for t, name, _ in index[-2:]:
            if t is not None:
                _need(t, torch.int32, name)
    for t, name in kv:
        if t.get_device() != dev or t.shape != (rows, heads, dim):
            raise PkvError(f"{name} must be [{rows}, {heads}, {dim}] on the current device")
    for t, name, least in index:
        if t is not None and (t.get_device() != dev or t.numel() < least):
            raise PkvError(f"{name} must have at least {least} entries, on the current device")
    if out.numel() != n * d or out.dtype is not torch.bfloat16 or out.get_device() != dev or not out.is_contiguous():
        raise PkvError("out must be contiguous bf16 like q")
    if lse.numel() != n or lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous():
        raise PkvError("lse must be contiguous fp32 [T, Hq]")
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise PkvError("the workspace must be contiguous, on the current device")


def paged_decode_attn(q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, cu_q=None,
                      reqs: Optional[Reqs] = None, scale=None, out=None, lse=None, workspace=None,
                      stream=None, k_scale=1.0, v_scale=1.0, window=None, sinks=0):
    """One query token per request against its paged context. q [T, Hq, D]. An FP8 cache is
    dequantised as it is read, with the per-tensor scales or with the scale of each block and KV
    head (k_scale, v_scale: fp32 tensors [num_blocks, Hkv]).

    With a window the token sees the last `window` keys, its own among them, and the first `sinks`
    keys; table entries of the blocks between them are not read."""
    lib = _lib.load()
    _need(q, torch.bfloat16, "q")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    T, Hq, D = q.shape
    R = seq_lens.numel()
    reqs = reqs or Reqs(max_reqs=R, batch_reqs=R)
    other = _other(stream)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, other)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, other)
    need = lib.pkv_paged_decode_workspace_size(reqs.max_reqs, Hq, cache.num_kv_heads, D, max_seq_len)
    win = _window(window, sinks)
    workspace = _scratch(need, workspace, q.device, other)
    if win is not None:
        batch, width = reqs.batch_reqs, block_tables.shape[1]
        index = ((block_tables, "block_tables", batch * width), (seq_lens, "seq_lens", batch), (k_cache, "the cache", 0))
        if cu_q is not None:
            _need(cu_q, torch.int32, "cu_q")
            index += ((cu_q, "cu_q", batch + 1),)
        elif reqs.order is None and T < min(reqs.max_reqs, batch):
            raise PkvError("q must have a row for each request")
        _window_args(q, 0, cache.head_dim, 0, reqs, index, out, lse, (), workspace)
        _check(lib.pkv_window_decode_attn(_ptr(q), cache, _ptr(block_tables), width,
                                          _ptr(seq_lens), _ptr(cu_q), reqs.c(), Hq, max_seq_len, *win,
                                          _scale(scale, D), _ptr(out), _ptr(lse), _ptr(workspace),
                                          need, _stream(stream)), "paged_decode_attn")
        return out, lse
    _check(lib.pkv_paged_decode_attn(_ptr(q), cache, _ptr(block_tables), block_tables.shape[1],
                                     _ptr(seq_lens), _ptr(cu_q), reqs.c(), Hq, max_seq_len,
                                     _scale(scale, D), _ptr(out), _ptr(lse), _ptr(workspace),
                                     need, _stream(stream)), "paged_decode_attn")
    return out, lse


def paged_decode_attn_noalloc(q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, out, lse,
                              cu_q=None, reqs: Optional[Reqs] = None, scale=None, stream=None,
                              k_scale=1.0, v_scale=1.0):
    """paged_decode_attn for callers that cannot allocate: the library uses its own fixed
    device scratch (NOALLOC_SCRATCH_BYTES per GPU) and the caller passes out and lse."""
    lib = _lib.load()
    _need(q, torch.bfloat16, "q")
    _need(out, torch.bfloat16, "out")
    _need(lse, torch.float32, "lse")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    T, Hq, D = q.shape
    R = seq_lens.numel()
    reqs = reqs or Reqs(max_reqs=R, batch_reqs=R)
    _check(lib.pkv_paged_decode_attn_noalloc(_ptr(q), cache, _ptr(block_tables), block_tables.shape[1],
                                             _ptr(seq_lens), _ptr(cu_q), reqs.c(), Hq, max_seq_len,
                                             _scale(scale, D), _ptr(out), _ptr(lse), _stream(stream)),
           "paged_decode_attn_noalloc")
    return out, lse


def mla_decode_attn(q, latent_cache, block_tables, seq_lens, max_seq_len, scale, v_dim=512, cu_q=None,
                    reqs: Optional[Reqs] = None, out=None, lse=None, workspace=None, stream=None):
    """Absorbed MLA decode. q [T, Hq, 576]; latent_cache [num_blocks, 16, 1, 576] bf16 (keys =
    all 576 dims of a token's latent row, values = its first v_dim). Returns out [T, Hq, v_dim]
    and lse [T, Hq]. The softmax scale is the model's (no default)."""
    lib = _lib.load()
    _need(q, torch.bfloat16, "q")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    cache = make_cache(latent_cache, latent_cache)
    T, Hq, Dk = q.shape
    R = seq_lens.numel()
    reqs = reqs or Reqs(max_reqs=R, batch_reqs=R)
    other = _other(stream)
    if out is None:
        out = _empty((T, Hq, v_dim), torch.bfloat16, q.device, other)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, other)
    need = lib.pkv_mla_decode_workspace_size(reqs.max_reqs, Hq, max_seq_len)
    workspace = _scratch(need, workspace, q.device, other)
    _check(lib.pkv_mla_decode_attn(_ptr(q), cache, _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
                                   _ptr(cu_q), reqs.c(), Hq, max_seq_len, float(scale), int(v_dim), _ptr(out),
                                   _ptr(lse), _ptr(workspace), need, _stream(stream)), "mla_decode_attn")
    return out, lse


def mla_decode_workspace_size(max_reqs, num_q_heads, max_seq_len) -> int:
    return int(_lib.load().pkv_mla_decode_workspace_size(max_reqs, num_q_heads, max_seq_len))


def extend_attn(q, k_new, v_new, cu_q, seq_lens, k_cache, v_cache, block_tables, max_q_len,
                max_seq_len, reqs: Optional[Reqs] = None, chunk_budget_tokens=32768, scale=None,
                out=None, lse=None, stream=None, k_scale=1.0, v_scale=1.0, workspace=None, window=None, sinks=0):
    """New tokens attend to their cached context (paged) and causally to themselves. An FP8
    cache (uint8 / float8 codes with per-tensor scales) is read as codes and converted in the
    kernel at head_dim 128; at head_dim 64 it is gathered into a bf16 workspace of the set's
    context first (allocated here when not given). k_scale / v_scale may be fp32 tensors
    [num_blocks, Hkv], a scale for each block and KV head (head_dim 128); the workspace then holds the
    partial results of contexts that are cut (allocated here when not given).

    With a window each row sees the last `window` keys up to its own and the first `sinks` keys (a
    bf16 cache, or an FP8 one with per-tensor scales at head_dim 128); table entries of blocks that no row sees
    are not read. Over FP8 the workspace holds what requests of many new tokens see, converted once (allocated
    here when not given)."""
    lib = _lib.load()
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new")):
        _need(t, torch.bfloat16, n)
    _need(cu_q, torch.int32, "cu_q")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(block_tables, torch.int32, "block_tables")
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    T, Hq, D = q.shape
    R = seq_lens.numel()
    reqs = reqs or Reqs(max_reqs=R, batch_reqs=R)
    other = _other(stream)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, other)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, other)
    win = _window(window, sinks)
    if win is not None:
        batch = reqs.batch_reqs
        _window_args(q, cache.num_kv_heads, cache.head_dim, T, reqs,
                     ((block_tables, "block_tables", batch * block_tables.shape[1]), (seq_lens, "seq_lens", batch),
                      (cu_q, "cu_q", batch + 1), (k_cache, "the cache", 0)), out, lse, ((k_new, "k_new"), (v_new, "v_new")), workspace)
        need = window_extend_workspace_size(T, reqs.max_reqs, max_q_len, max_seq_len, Hq, cache.num_kv_heads, D, *win,
                                            kv_dtype=cache.kv_dtype) if cache.kv_dtype == _lib.KV_FP8_E4M3 else 0
        workspace = _scratch(need, workspace, q.device, other)
        _check(lib.pkv_window_extend_attn(_ptr(q), _ptr(k_new), _ptr(v_new), T, _ptr(cu_q), _ptr(seq_lens), cache,
                                          _ptr(block_tables), block_tables.shape[1], reqs.c(), Hq, max_q_len,
                                          max_seq_len, *win, _scale(scale, D), _ptr(out), _ptr(lse),
                                          _ptr(workspace) if need else None, need, _stream(stream)), "extend_attn")
        return out, lse
    need = 0
    if cache.kv_dtype == _lib.KV_FP8_E4M3:
        need = extend_fp8_workspace_size(reqs.max_reqs, reqs.batch_reqs, max_seq_len, block_tables.shape[1],
                                         cache.num_kv_heads, cache.head_dim)
    elif cache.kv_dtype == _lib.KV_FP8_E4M3_BLOCK:
        need = extend_block_workspace_size(max_q_len, max_seq_len, Hq, cache.num_kv_heads)
    workspace = _scratch(need, workspace, q.device, other)
    _check(lib.pkv_extend_attn(_ptr(q), _ptr(k_new), _ptr(v_new), T, _ptr(cu_q), _ptr(seq_lens), cache,
                               _ptr(block_tables), block_tables.shape[1], reqs.c(), Hq, max_q_len,
                               max_seq_len, chunk_budget_tokens, _scale(scale, D), _ptr(out),
                               _ptr(lse), _ptr(workspace) if need else None, need, _stream(stream)), "extend_attn")
    return out, lse


def extend_block_workspace_size(max_q_len, max_seq_len, num_q_heads, num_kv_heads) -> int:
    return int(_lib.load().pkv_extend_block_workspace_size(max_q_len, max_seq_len, num_q_heads, num_kv_heads))


def window_extend_workspace_size(num_tokens, max_reqs, max_q_len, max_seq_len, num_q_heads, num_kv_heads, head_dim, window,
                                 sinks=0, kv_dtype=_lib.KV_FP8_E4M3) -> int:
    return int(_lib.load().pkv_window_extend_workspace_size(num_tokens, max_reqs, max_q_len, max_seq_len, num_q_heads,
                                                            num_kv_heads, head_dim, kv_dtype, *_window(window, sinks)))


def extend_fp8_workspace_size(max_reqs, batch_reqs, max_seq_len, max_blocks, num_kv_heads, head_dim) -> int:
    return int(_lib.load().pkv_extend_fp8_workspace_size(max_reqs, batch_reqs, max_seq_len, max_blocks,
                                                         num_kv_heads, head_dim))


def varlen_prefill_attn(q, k, v, cu_seqlens, max_seqlen, reqs: Optional[Reqs] = None, scale=None,
                        out=None, lse=None, stream=None, window=None, sinks=0):
    """Causal attention over packed variable-length prompts. With a window each row sees the last
    `window` keys up to its own and the first `sinks` keys of its prompt."""
    lib = _lib.load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    R = cu_seqlens.numel() - 1
    reqs = reqs or Reqs(max_reqs=R, batch_reqs=R)
    other = _other(stream)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, other)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, other)
    win = _window(window, sinks)
    if win is not None:
        _window_args(q, Hkv, D, T, reqs, ((cu_seqlens, "cu_seqlens", reqs.batch_reqs + 1),), out, lse, ((k, "k"), (v, "v")))
        _check(lib.pkv_window_prefill_attn(_ptr(q), _ptr(k), _ptr(v), T, _ptr(cu_seqlens), reqs.c(), Hq, Hkv, D,
                                           max_seqlen, *win, _scale(scale, D), _ptr(out), _ptr(lse),
                                           _stream(stream)), "varlen_prefill_attn")
        return out, lse
    _check(lib.pkv_varlen_prefill_attn(_ptr(q), _ptr(k), _ptr(v), T, _ptr(cu_seqlens), reqs.c(), Hq,
                                       Hkv, D, max_seqlen, _scale(scale, D), _ptr(out), _ptr(lse),
                                       _stream(stream)), "varlen_prefill_attn")
    return out, lse


def device_errors(clear: bool = True, stream=None) -> int:
    """Synchronise the stream and return (then clear) the device error word."""
    lib = _lib.load()
    flags = ctypes.c_uint32(0)
    st = lib.pkv_device_errors(ctypes.byref(flags), 1 if clear else 0, _stream(stream))
    if st not in (0, 5):
        _check(st, "device_errors")
    return int(flags.value)


def launch_count(reset: bool = False) -> int:
    return int(_lib.load().pkv_launch_count(1 if reset else 0))
