"""Torch-facing wrappers of the C ABI: pointers, sizes and streams from torch
tensors, nothing else.  Every step of the cache write and the decode runs in
libkvq's CUDA kernels; these functions refuse CPU tensors."""

import torch

from . import _abi as A


def fmt_id(fmt):
    return fmt if isinstance(fmt, int) else A.kvq_format_from_string(fmt)


def _dev_ptr(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libkvq has no CPU path)")
    return t.data_ptr()


def _dtype_code(t, name):
    if t.dtype == torch.float32:
        return A.KVQ_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return A.KVQ_DTYPE_BF16
    raise ValueError(f"{name} must be float32 or bfloat16")


def _stream_ptr(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def block_bytes(fmt, side, block_size, num_kv_heads, head_dim):
    return A.kvq_block_bytes(fmt_id(fmt), side, block_size, num_kv_heads, head_dim)


def alloc_pool(num_blocks, fmt, side, block_size, num_kv_heads, head_dim, device="cuda",
               stride=None):
    """uint8 [num_blocks, stride] pool for one side; stride rounded up to 16 bytes."""
    b = block_bytes(fmt, side, block_size, num_kv_heads, head_dim)
    stride = stride or (b + 15) // 16 * 16
    return torch.zeros((num_blocks, stride), dtype=torch.uint8, device=device)


def cache_write(key, value, k_cache, v_cache, slot_mapping, fmt, num_kv_heads, head_dim,
                block_size, key_stride=None, value_stride=None, k_scale=1.0, v_scale=1.0,
                num_blocks=None, error_flag=None, stream=None, num_tokens=None):
    """Write rows of ``key``/``value`` (first element of token 0, head 0 at
    ``key.data_ptr()``) into the pools ``k_cache``/``v_cache`` ([num_blocks,
    stride] uint8) at ``slot_mapping`` (int64)."""
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    n = slot_mapping.numel() if num_tokens is None else num_tokens
    kd = _dtype_code(key, "key")
    if _dtype_code(value, "value") != kd:
        raise ValueError("key and value must share a dtype")
    ks = key_stride if key_stride is not None else key.stride(0)
    vs = value_stride if value_stride is not None else value.stride(0)
    nb = k_cache.shape[0] if num_blocks is None else num_blocks
    A.kvq_cache_write(
        _dev_ptr(key, "key"), _dev_ptr(value, "value"), kd, _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(slot_mapping, "slot_mapping"), n, nb,
        num_kv_heads, head_dim, block_size, ks, vs, k_cache.stride(0), v_cache.stride(0),
        float(k_scale), float(v_scale), fmt_id(fmt), _dev_ptr(error_flag, "error_flag"),
        _stream_ptr(stream))


def decode_kernel(fmt, head_dim, num_kv_heads, block_size):
    """Name of the decode kernel paged_decode launches on the current device
    for these arguments ("decode_tma_kernel" or "decode_tc_kernel")."""
    p = A.kvq_decode_path(fmt_id(fmt), head_dim, num_kv_heads, block_size)
    if p < 0:
        raise ValueError("arguments the decode rejects")
    return "decode_tma_kernel" if p == 1 else "decode_tc_kernel"


def decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           max_blocks_per_seq, sliding_window, fmt):
    return A.kvq_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                        block_size, max_blocks_per_seq, sliding_window,
                                        fmt_id(fmt))


def alloc_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                    max_blocks_per_seq, sliding_window, fmt, device="cuda"):
    n = decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                               max_blocks_per_seq, sliding_window, fmt)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def paged_decode(q, k_cache, v_cache, block_tables, seq_lens, fmt, num_kv_heads,
                 block_size, out=None, out_dtype=torch.float32, sm_scale=0.0, k_scale=1.0,
                 v_scale=1.0, sliding_window=0, sparse_v_threshold=0.0, workspace=None,
                 num_blocks=None, error_flag=None, stream=None):
    """Decode attention: q [num_seqs, num_q_heads, head_dim] (row stride q.stride(0)),
    block_tables int32 [num_seqs, max_blocks], seq_lens int32 [num_seqs]."""
    num_seqs, nq, hd = q.shape
    if q.stride(2) != 1 or q.stride(1) != hd:
        raise ValueError("q heads must be contiguous [.., num_q_heads, head_dim]")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    if not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous")
    mb = block_tables.shape[1]
    if out is None:
        out = torch.empty((num_seqs, nq, hd), dtype=out_dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(num_seqs, nq, num_kv_heads, hd, block_size, mb,
                                    sliding_window, fmt, device=q.device)
    nb = k_cache.shape[0] if num_blocks is None else num_blocks
    A.kvq_paged_decode(
        _dev_ptr(q, "q"), _dtype_code(q, "q"), q.stride(0), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(out, "out"), _dtype_code(out, "out"),
        _dev_ptr(block_tables, "block_tables"), mb, _dev_ptr(seq_lens, "seq_lens"), num_seqs,
        nb, nq, num_kv_heads, hd, block_size, k_cache.stride(0), v_cache.stride(0),
        float(sm_scale), float(k_scale), float(v_scale), int(sliding_window),
        float(sparse_v_threshold), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), fmt_id(fmt),
        _dev_ptr(error_flag, "error_flag"), _stream_ptr(stream))
    return out


def paged_prefill(q, cu_q, max_chunk, k_cache, v_cache, block_tables, seq_lens, fmt,
                  num_kv_heads, block_size, out=None, out_dtype=torch.float32, sm_scale=0.0,
                  k_scale=1.0, v_scale=1.0, sliding_window=0, num_blocks=None, error_flag=None,
                  stream=None):
    """Chunked-prefill attention: q [total_q, num_q_heads, head_dim] (row stride
    q.stride(0)), cu_q int32 [num_seqs + 1] query offsets per sequence, the last
    cu_q[s+1] - cu_q[s] of sequence s's seq_lens[s] cached positions being its
    queries (causal)."""
    total_q, nq, hd = q.shape
    if q.stride(2) != 1 or q.stride(1) != hd:
        raise ValueError("q heads must be contiguous [.., num_q_heads, head_dim]")
    for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (cu_q, "cu_q")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
    num_seqs = seq_lens.shape[0]
    mb = block_tables.shape[1]
    if out is None:
        out = torch.empty((total_q, nq, hd), dtype=out_dtype, device=q.device)
    nb = k_cache.shape[0] if num_blocks is None else num_blocks
    A.kvq_paged_prefill(
        _dev_ptr(q, "q"), _dtype_code(q, "q"), q.stride(0), _dev_ptr(cu_q, "cu_q"),
        int(max_chunk), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
        _dev_ptr(out, "out"), _dtype_code(out, "out"), _dev_ptr(block_tables, "block_tables"),
        mb, _dev_ptr(seq_lens, "seq_lens"), num_seqs, nb, nq, num_kv_heads, hd, block_size,
        k_cache.stride(0), v_cache.stride(0), float(sm_scale), float(k_scale), float(v_scale),
        int(sliding_window), fmt_id(fmt), _dev_ptr(error_flag, "error_flag"),
        _stream_ptr(stream))
    return out


# ------------------------------------------------- prompts, shared prefixes, eviction
#
# These run on the device of their tensors whatever the current device is, and
# allocate what they return (and their workspace, if none is given) for the
# stream the work is queued on.

class _on:
    """The tensors' one device as current, with `stream` (default: that
    device's current stream) current on it; gives the stream's address.
    (Switching device and stream costs more host time than the launches of a
    small call, so nothing is switched where both are current already.)"""

    __slots__ = ("ptr", "contexts")

    def __init__(self, stream, **tensors):
        dev, first = -1, None
        for name, t in tensors.items():
            if t is None:
                continue
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor (libkvq has no CPU path)")
            d = t.get_device()
            if dev < 0:
                dev, first = d, name
            elif d != dev:
                raise ValueError(f"{name} is on cuda:{d}, {first} on cuda:{dev}")
        if stream is not None and stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
        self.contexts = ()
        here = dev == torch.cuda.current_device()
        s = torch.cuda.current_stream(dev) if stream is None else stream
        if not here:
            self.contexts = (torch.cuda.device(dev), torch.cuda.stream(s))
        elif stream is not None and stream != torch.cuda.current_stream():
            self.contexts = (torch.cuda.stream(s),)
        self.ptr = s.cuda_stream

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _int32(t, name, *shape):
    """A contiguous int32 tensor, of the given shape where one is given."""
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32")
    if shape and (t.dim() != len(shape) or
                  any(w is not None and w != g for w, g in zip(shape, t.shape))):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _heads(t, name):
    """[tokens, heads, head_dim] with contiguous heads and any token stride."""
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1) or \
            (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} heads must be contiguous [.., heads, head_dim]")
    # a tensor of one token has no meaningful token stride
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] * t.shape[2])


def _pool(t, name):
    if t.dtype != torch.uint8 or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be uint8 [num_blocks, bytes] with contiguous blocks")
    return t.stride(0)


def _pages(t, name, num_blocks):
    nb = t.shape[0] if num_blocks is None else num_blocks
    if nb < 1 or nb > t.shape[0]:
        raise ValueError(f"num_blocks must be in [1, {t.shape[0]}] ({name}'s blocks)")
    return nb


def _flag(t):
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1):
        raise ValueError("error_flag must be int32")


def _out(out, shape, dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if tuple(out.shape) != tuple(shape) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {tuple(shape)}")
    return out


def prompt_attention(q, k, v, cu_seqlens, max_seqlen, out=None, out_dtype=torch.float32,
                     sm_scale=0.0, sliding_window=0, lse=None, error_flag=None, stream=None):
    """Causal attention over whole prompts packed one after another, from the
    rows a layer has just computed: q [tokens, num_q_heads, head_dim], k and v
    [tokens, num_kv_heads, head_dim] (token strides are free: views of a fused
    QKV row), cu_seqlens int32 [num_seqs + 1].  ``lse``: optional fp32
    [tokens, num_q_heads] that receives log of the softmax denominators."""
    total, nq, hd = q.shape
    qs, ks, vs = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    if k.shape != v.shape or k.shape[0] != total or k.shape[2] != hd:
        raise ValueError("k and v must be [tokens, num_kv_heads, head_dim] like q")
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k and v must share a dtype")
    _int32(cu_seqlens, "cu_seqlens")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [num_seqs + 1]")
    _flag(error_flag)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (total, nq) or
                            not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [tokens, num_q_heads]")
    with _on(stream, q=q, k=k, v=v, cu_seqlens=cu_seqlens, out=out, lse=lse,
             error_flag=error_flag) as st:
        out = _out(out, q.shape, out_dtype, q.device)
        A.kvq_prompt_attention(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q, "q"), qs, ks, vs,
            cu_seqlens.data_ptr(), total, int(max_seqlen), out.data_ptr(),
            _dtype_code(out, "out"), _dev_ptr(lse, "lse"), cu_seqlens.shape[0] - 1, nq,
            k.shape[1], hd, float(sm_scale), int(sliding_window),
            _dev_ptr(error_flag, "error_flag"), st)
    return out


def shared_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size,
                           max_prefix_blocks, max_blocks_per_seq, sliding_window, fmt):
    return A.kvq_shared_decode_workspace_bytes(
        num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size, max_prefix_blocks,
        max_blocks_per_seq, sliding_window, fmt_id(fmt))


def alloc_shared_workspace(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size,
                           max_prefix_blocks, max_blocks_per_seq, sliding_window, fmt,
                           device="cuda"):
    """Workspace of paged_decode_shared (any content; one per call in flight)."""
    with torch.cuda.device(device):
        n = shared_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim,
                                   block_size, max_prefix_blocks, max_blocks_per_seq,
                                   sliding_window, fmt)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def paged_decode_shared(q, k_cache, v_cache, prefix_tables, prefix_lens, cu_groups, block_tables,
                        seq_lens, fmt, num_kv_heads, block_size, out=None,
                        out_dtype=torch.float32, sm_scale=0.0, k_scale=1.0, v_scale=1.0,
                        sliding_window=0, workspace=None, num_blocks=None, error_flag=None,
                        stream=None):
    """Decode of a batch in groups that share a prefix: sequences
    cu_groups[g] .. cu_groups[g + 1] - 1 attend to the prefix_lens[g] positions
    in prefix_tables[g], then to their own seq_lens[s] in block_tables[s]."""
    num_seqs, nq, hd = q.shape
    qs = _heads(q, "q")
    _int32(prefix_lens, "prefix_lens")
    num_groups = prefix_lens.shape[0]
    _int32(prefix_tables, "prefix_tables", num_groups, None)
    _int32(cu_groups, "cu_groups", num_groups + 1)
    _int32(block_tables, "block_tables", num_seqs, None)
    _int32(seq_lens, "seq_lens", num_seqs)
    kst, vst = _pool(k_cache, "k_cache"), _pool(v_cache, "v_cache")
    nb = min(_pages(k_cache, "k_cache", num_blocks), _pages(v_cache, "v_cache", num_blocks))
    _flag(error_flag)
    with _on(stream, q=q, k_cache=k_cache, v_cache=v_cache, prefix_tables=prefix_tables,
             prefix_lens=prefix_lens, cu_groups=cu_groups, block_tables=block_tables,
             seq_lens=seq_lens, out=out, workspace=workspace, error_flag=error_flag) as st:
        out = _out(out, q.shape, out_dtype, q.device)
        mp, mb = prefix_tables.shape[1], block_tables.shape[1]
        if workspace is None:
            workspace = alloc_shared_workspace(num_seqs, num_groups, nq, num_kv_heads, hd,
                                               block_size, mp, mb, sliding_window, fmt,
                                               device=q.device)
        A.kvq_paged_decode_shared(
            q.data_ptr(), _dtype_code(q, "q"), qs, k_cache.data_ptr(), v_cache.data_ptr(),
            out.data_ptr(), _dtype_code(out, "out"), prefix_tables.data_ptr(), mp,
            prefix_lens.data_ptr(), cu_groups.data_ptr(), num_groups, block_tables.data_ptr(), mb,
            seq_lens.data_ptr(), num_seqs, nb, nq, num_kv_heads, hd, block_size, kst, vst,
            float(sm_scale), float(k_scale), float(v_scale), int(sliding_window),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), fmt_id(fmt),
            _dev_ptr(error_flag, "error_flag"), st)
    return out


def mass_workspace_bytes(total_q, num_seqs, max_chunk, num_q_heads, num_kv_heads, block_size,
                         max_blocks_per_seq):
    return A.kvq_attention_mass_workspace_bytes(total_q, num_seqs, max_chunk, num_q_heads,
                                                num_kv_heads, block_size, max_blocks_per_seq)


def alloc_mass_workspace(total_q, num_seqs, max_chunk, num_q_heads, num_kv_heads, block_size,
                         max_blocks_per_seq, device="cuda"):
    """Workspace of attention_mass (any content; one per call in flight).  It also
    serves calls with fewer queries and the other arguments the same."""
    with torch.cuda.device(device):
        n = mass_workspace_bytes(total_q, num_seqs, max_chunk, num_q_heads, num_kv_heads,
                                 block_size, max_blocks_per_seq)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _mass_rows(t, name, num_seqs, num_kv_heads):
    """fp32 [num_seqs, num_kv_heads, columns], rows evenly spaced."""
    if t.dtype != torch.float32 or t.dim() != 3 or tuple(t.shape[:2]) != (num_seqs, num_kv_heads) \
            or t.shape[2] < 1 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be float32 [num_seqs, num_kv_heads, positions]")
    row = t.stride(1) if num_kv_heads > 1 else t.stride(0) if num_seqs > 1 else t.shape[2]
    if row < t.shape[2] or (num_seqs > 1 and t.stride(0) != row * num_kv_heads):
        raise ValueError(f"{name} rows must be evenly spaced")
    return row


def attention_mass(q, cu_q, max_chunk, k_cache, block_tables, seq_lens, fmt, num_kv_heads,
                   block_size, mass_in=None, mass_out=None, sm_scale=0.0, k_scale=1.0,
                   sliding_window=0, workspace=None, num_blocks=None, error_flag=None,
                   stream=None):
    """Adds the softmax weights that the chunk's queries (the last
    cu_q[s + 1] - cu_q[s] positions of sequence s, as in paged_prefill) give
    each cached position, summed over the query heads of a kv head:
    mass_out[s, h, t] = mass_in[s, h, t] + weights, t < seq_lens[s].
    ``mass_in`` None counts as zeros; ``mass_out`` None is allocated (zeros,
    max_blocks * block_size positions); they may be the same tensor."""
    total_q, nq, hd = q.shape
    qs = _heads(q, "q")
    _int32(seq_lens, "seq_lens")
    num_seqs = seq_lens.shape[0]
    _int32(cu_q, "cu_q", num_seqs + 1)
    _int32(block_tables, "block_tables", num_seqs, None)
    kst = _pool(k_cache, "k_cache")
    nb = _pages(k_cache, "k_cache", num_blocks)
    mb = block_tables.shape[1]
    _flag(error_flag)
    with _on(stream, q=q, cu_q=cu_q, k_cache=k_cache, block_tables=block_tables, seq_lens=seq_lens,
             mass_in=mass_in, mass_out=mass_out, workspace=workspace, error_flag=error_flag) as st:
        if mass_out is None:
            mass_out = torch.zeros((num_seqs, num_kv_heads, mb * block_size), device=q.device)
        os_ = _mass_rows(mass_out, "mass_out", num_seqs, num_kv_heads)
        is_ = 0
        if mass_in is not None:
            is_ = _mass_rows(mass_in, "mass_in", num_seqs, num_kv_heads)
            if mass_in.shape[2] < mass_out.shape[2]:
                raise ValueError("mass_in has fewer positions than mass_out")
            if mass_in.data_ptr() == mass_out.data_ptr() and is_ != os_:
                raise ValueError("mass_in and mass_out overlap")
        if mass_out.shape[2] < os_ and num_seqs * num_kv_heads > 0:
            # columns between rows are not the caller's to overwrite
            if mass_out.shape[2] < mb * block_size:
                raise ValueError("mass_out must hold max_blocks * block_size positions, or be contiguous")
        if workspace is None:
            workspace = alloc_mass_workspace(total_q, num_seqs, max_chunk, nq, num_kv_heads,
                                             block_size, mb, device=q.device)
        A.kvq_attention_mass(
            q.data_ptr(), _dtype_code(q, "q"), qs, cu_q.data_ptr(), total_q, int(max_chunk),
            k_cache.data_ptr(), block_tables.data_ptr(), mb, seq_lens.data_ptr(), num_seqs, nb, nq,
            num_kv_heads, hd, block_size, kst, float(sm_scale), float(k_scale),
            int(sliding_window), _dev_ptr(mass_in, "mass_in"), is_, mass_out.data_ptr(), os_,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), fmt_id(fmt),
            _dev_ptr(error_flag, "error_flag"), st)
    return mass_out


def evict_select(mass, seq_lens, keep, sink=0, recent=0, kept=None, new_lens=None,
                 error_flag=None, stream=None):
    """(kept, new_lens): per (sequence, kv head) the ascending positions of the
    first ``sink``, the last ``recent`` and the largest other entries of
    ``mass`` [num_seqs, num_kv_heads, positions], ``keep`` in all; kept int32
    [num_seqs, num_kv_heads, keep], -1 past new_lens[s] = min(seq_lens[s], keep)."""
    num_seqs, nkv, _ = mass.shape
    ms = _mass_rows(mass, "mass", num_seqs, nkv)
    _int32(seq_lens, "seq_lens", num_seqs)
    keep = int(keep)
    if keep < 1:
        raise ValueError("keep must be >= 1")
    if ms != mass.shape[2] and num_seqs * nkv > 1:
        raise ValueError("mass must be contiguous (its row length bounds the positions)")
    _flag(error_flag)
    for t, name, shape in ((kept, "kept", (num_seqs, nkv, keep)), (new_lens, "new_lens", (num_seqs,))):
        if t is not None:
            _int32(t, name, *shape)
    if new_lens is not None and new_lens.data_ptr() == seq_lens.data_ptr() and num_seqs:
        raise ValueError("new_lens must not be seq_lens")
    with _on(stream, mass=mass, seq_lens=seq_lens, kept=kept, new_lens=new_lens,
             error_flag=error_flag) as st:
        if kept is None:
            kept = torch.empty((num_seqs, nkv, keep), dtype=torch.int32, device=mass.device)
        if new_lens is None:
            new_lens = torch.empty((num_seqs,), dtype=torch.int32, device=mass.device)
        A.kvq_evict_select(
            mass.data_ptr(), mass.shape[2], seq_lens.data_ptr(), num_seqs, nkv, keep, int(sink),
            int(recent), kept.data_ptr(), new_lens.data_ptr(), _dev_ptr(error_flag, "error_flag"),
            st)
    return kept, new_lens


def cache_compact(k_cache, v_cache, block_tables, seq_lens, kept, fmt, num_kv_heads, head_dim,
                  block_size, dst_tables=None, mass=None, mass_out=None, num_blocks=None,
                  error_flag=None, stream=None):
    """Moves row (kept[s, h, i], h) of each sequence to position i on both
    sides, within the sequence's own pages, or to the pages of ``dst_tables``
    int32 [num_seqs, max_dst_blocks].  ``mass`` (moved with the rows, if
    given): within itself, or into ``mass_out``; needed for other pages."""
    _int32(seq_lens, "seq_lens")
    num_seqs = seq_lens.shape[0]
    _int32(block_tables, "block_tables", num_seqs, None)
    _int32(kept, "kept", num_seqs, num_kv_heads, None)
    if dst_tables is not None:
        _int32(dst_tables, "dst_tables", num_seqs, None)
    kst, vst = _pool(k_cache, "k_cache"), _pool(v_cache, "v_cache")
    nb = min(_pages(k_cache, "k_cache", num_blocks), _pages(v_cache, "v_cache", num_blocks))
    _flag(error_flag)
    keep = kept.shape[2]
    is_ = os_ = 0
    if mass is not None:
        if mass_out is None:
            mass_out = mass
        is_ = _mass_rows(mass, "mass", num_seqs, num_kv_heads)
        os_ = _mass_rows(mass_out, "mass_out", num_seqs, num_kv_heads)
        if mass.shape[2] < block_tables.shape[1] * block_size or mass_out.shape[2] < keep:
            raise ValueError("mass must hold max_blocks * block_size positions, mass_out keep")
    elif mass_out is not None:
        raise ValueError("mass_out without mass")
    with _on(stream, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
             seq_lens=seq_lens, kept=kept, dst_tables=dst_tables, mass=mass, mass_out=mass_out,
             error_flag=error_flag) as st:
        A.kvq_cache_compact(
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
            block_tables.shape[1], seq_lens.data_ptr(), kept.data_ptr(), keep,
            _dev_ptr(dst_tables, "dst_tables"), 0 if dst_tables is None else dst_tables.shape[1],
            num_seqs, nb, num_kv_heads, head_dim, block_size, kst, vst, _dev_ptr(mass, "mass"),
            is_, _dev_ptr(mass_out, "mass_out"), os_, fmt_id(fmt),
            _dev_ptr(error_flag, "error_flag"), st)
