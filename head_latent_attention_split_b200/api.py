"""torch-tensor front end of the C ABI: shape/dtype inference and output allocation."""
from __future__ import annotations

from . import binding as _b


def _dtype_code(t, what):
    import torch
    if t.dtype == torch.float32:
        return _b.F32
    if t.dtype == torch.bfloat16:
        return _b.BF16
    if t.dtype in (torch.uint8, getattr(torch, "float8_e4m3fn", None)):
        return _b.E4M3
    raise TypeError(f"{what}: unsupported dtype {t.dtype}")


def params_for(q_lat, q_rope, kv_cache, block_table, softmax_scale, causal=False, out_dtype=None,
               num_workers=0, kernel="auto") -> _b.Params:
    """Build mla_decode_params_t from tensor shapes.

    q_lat [B, Sq, H, r], q_rope [B, Sq, H, d_r], kv_cache [num_blocks, block_size, r + d_r]
    (f32 / bf16) or e4m3 codes [num_blocks, block_size, r], block_table [B, max_blocks].
    """
    B, Sq, H, r = q_lat.shape
    d_r = q_rope.shape[-1] if q_rope is not None else 0
    qd = _dtype_code(q_lat, "q_lat")
    cd = _dtype_code(kv_cache, "kv_cache")
    od = qd if out_dtype is None else out_dtype
    nb, bs = kv_cache.shape[0], kv_cache.shape[1]
    return _b.make_params(B, Sq, H, r, d_r, bs, nb, block_table.shape[1], qd, cd, od, causal, softmax_scale,
                          num_workers, kernel)


def decode(q_lat, q_rope, kv_cache, block_table, seq_lens, softmax_scale, causal=False, k_rope_cache=None,
           kv_scale=None, out=None, lse=None, workspace=None, out_dtype=None, num_workers=0, kernel="auto",
           stream=None):
    """One MLA decode step on the current CUDA device. Returns (out, lse).

    out [B, Sq, H, r] (dtype of q unless out_dtype), lse [B, Sq, H] float32 (natural log).
    """
    import torch
    p = params_for(q_lat, q_rope, kv_cache, block_table, softmax_scale, causal, out_dtype, num_workers, kernel)
    dev = q_lat.device
    if out is None:
        od = {_b.F32: torch.float32, _b.BF16: torch.bfloat16}[p.out_dtype]
        out = torch.empty(q_lat.shape, dtype=od, device=dev)
    if lse is None:
        lse = torch.empty(q_lat.shape[:3], dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(_b.workspace_size(p), 1), dtype=torch.uint8, device=dev)
    _b.mla_decode(p, q_lat, q_rope, kv_cache, k_rope_cache, kv_scale, block_table, seq_lens, out, lse, workspace,
                  stream=stream)
    return out, lse


def decode_host_io(q_lat_host, q_rope_host, kv_cache, block_table_host, seq_lens_host, softmax_scale,
                   causal=False, k_rope_cache=None, kv_scale=None, out_host=None, lse_host=None, workspace=None,
                   out_dtype=None, num_workers=0, kernel="auto", stream=None):
    """Decode step with per-step tensors in pinned host memory (see mla_decode_host_io)."""
    import torch
    p = params_for(q_lat_host, q_rope_host, kv_cache, block_table_host, softmax_scale, causal, out_dtype,
                   num_workers, kernel)
    if out_host is None:
        od = {_b.F32: torch.float32, _b.BF16: torch.bfloat16}[p.out_dtype]
        out_host = torch.empty(q_lat_host.shape, dtype=od, pin_memory=True)
    if lse_host is None:
        lse_host = torch.empty(q_lat_host.shape[:3], dtype=torch.float32, pin_memory=True)
    if workspace is None:
        workspace = torch.empty(_b.host_io_workspace_size(p), dtype=torch.uint8, device=kv_cache.device)
    _b.mla_decode_host_io(p, q_lat_host, q_rope_host, kv_cache, k_rope_cache, kv_scale, block_table_host,
                          seq_lens_host, out_host, lse_host, workspace, stream=stream)
    return out_host, lse_host


def cache_append(c_new, k_rope_new, kv_cache, block_table, seq_lens, k_rope_cache=None, kv_scale=None,
                 rope=False, rope_base=10000.0, stream=None):
    """Write the Sq new tokens of each sequence into the paged cache (see mla_cache_append).

    c_new [B, Sq, r] and k_rope_new [B, Sq, d_r] (float32 for an f32 cache, bf16 otherwise);
    kv_cache [num_blocks, block_size, r + d_r] (f32 / bf16), or e4m3 codes
    [num_blocks, block_size, r] (uint8) with k_rope_cache bf16 [num_blocks, block_size, d_r]
    and kv_scale float32 [num_blocks, block_size]. Token s of sequence b lands at position
    seq_lens[b] - Sq + s. With rope, the RoPE key is rotated for that position first (not for a cache that
    cache_compact has cut: its kept keys have the rotations of the whole sequence, so rotate the new ones for
    their places there and leave rope off).
    """
    B, Sq, r = c_new.shape
    d_r = k_rope_new.shape[-1] if k_rope_new is not None else 0
    p = _b.make_append_params(B, Sq, r, d_r, kv_cache.shape[1], kv_cache.shape[0], block_table.shape[1],
                              _dtype_code(c_new, "c_new"), _dtype_code(kv_cache, "kv_cache"), rope, rope_base)
    _b.mla_cache_append(p, c_new, k_rope_new, kv_cache, k_rope_cache, kv_scale, block_table, seq_lens, stream=stream)


def head_gemm(x, w, y=None, stream=None):
    """y[m, h, :] = x[m, h, :] @ w[h] on the tensor cores (bf16 in and out, fp32 accumulation).

    x [rows, H, k] (or [B, Sq, H, k]), w [H, k, n]; k and n multiples of 64. Query absorption:
    head_gemm(q_nope, W_UK) -> q_lat; output projection: head_gemm(out, W_UV.transpose(1, 2)).
    """
    import torch
    lead = x.shape[:-2]
    H, k = x.shape[-2], x.shape[-1]
    n = w.shape[-1]
    rows = int(x.numel() // (H * k))
    if y is None:
        y = torch.empty((*lead, H, n), dtype=torch.bfloat16, device=x.device)
    p = _b.HeadGemmParams(rows=rows, heads=H, k=k, n=n, reserved=0)
    _b.mla_head_gemm(p, x, w, y, stream=stream)
    return y


def dsa_params_for(q_codes, k_codes, block_table, max_seq_len, top_k, causal=False) -> _b.DsaParams:
    """mla_dsa_params_t from tensor shapes: q_codes [B, Sq, H^I, d^I], k_codes
    [num_blocks, block_size, d^I], block_table [B, max_blocks]."""
    B, Sq, HI, dI = q_codes.shape
    nb, bs = k_codes.shape[0], k_codes.shape[1]
    return _b.make_dsa_params(B, Sq, HI, dI, bs, nb, block_table.shape[1], max_seq_len, top_k, causal)


def dsa_index(q_codes, q_scale, weights, k_codes, k_scale, block_table, seq_lens, max_seq_len, scores=None,
              causal=False, stream=None):
    """Lightning-indexer scores [B, Sq, max_seq_len] float32 (see mla_dsa_index). Code
    tensors are uint8 (or float8_e4m3fn) e4m3 codes."""
    import torch
    p = dsa_params_for(q_codes, k_codes, block_table, max_seq_len, 1, causal)
    if scores is None:
        scores = torch.empty((q_codes.shape[0], q_codes.shape[1], max_seq_len), dtype=torch.float32,
                             device=q_codes.device)
    _b.mla_dsa_index(p, q_codes, q_scale, weights, k_codes, k_scale, block_table, seq_lens, scores, stream=stream)
    return scores


def dsa_topk(scores, seq_lens, top_k, causal=False, indices=None, counts=None, stream=None):
    """Top-k positions per query row: (indices int32 [B, Sq, top_k] ascending, -1 padded;
    counts int32 [B, Sq]) (see mla_dsa_topk)."""
    import torch
    B, Sq, max_seq_len = scores.shape
    p = _b.make_dsa_params(B, Sq, 64, 128, 64, 1, max(1, (max_seq_len + 63) // 64), max_seq_len, top_k, causal)
    if indices is None:
        indices = torch.empty((B, Sq, top_k), dtype=torch.int32, device=scores.device)
    if counts is None:
        counts = torch.empty((B, Sq), dtype=torch.int32, device=scores.device)
    _b.mla_dsa_topk(p, scores, seq_lens, indices, counts, stream=stream)
    return indices, counts


def sparse_decode(q_lat, q_rope, kv_cache, block_table, indices, counts, softmax_scale, out=None, lse=None,
                  workspace=None, num_workers=0, stream=None, kernel="auto"):
    """MLA decode over selected positions (q_len 1, bf16 cache): indices [B, top_k] (or
    [B, 1, top_k]) int32, counts [B] (or [B, 1]) int32. Returns (out, lse)."""
    import torch
    p = params_for(q_lat, q_rope, kv_cache, block_table, softmax_scale, False, None, num_workers, kernel)
    top_k = indices.shape[-1]
    dev = q_lat.device
    if out is None:
        out = torch.empty(q_lat.shape, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(q_lat.shape[:3], dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(_b.workspace_size(p), 1), dtype=torch.uint8, device=dev)
    _b.mla_sparse_decode(p, top_k, q_lat, q_rope, kv_cache, block_table, indices, counts, out, lse, workspace,
                         stream=stream)
    return out, lse


# ---------------------------------------------------------------- window decode, eviction, draft verification
#
# The calls below check their tensors (device, type, shape, contiguity) before the library sees a
# pointer, run on the tensors' device whatever the current one is, and allocate on the stream
# they launch on. A small call's kernels take a few microseconds, so the checks are one expression
# per tensor, the argument structures are filled by position, and new tensors come from empty_like and
# empty_strided (1.3 and 1.4 us a call where torch.empty takes 2.2).
def _raw_stream(dev):
    """Handle of dev's current stream."""
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(dev.index)   # torch.cuda.current_stream without the object
    except AttributeError:
        return torch.cuda.current_stream(dev).cuda_stream


def _away(dev, stream):
    """None when the call can run as it stands (on dev's current stream, dev current), else a context that
    makes dev and `stream` (a torch stream or a raw handle) current."""
    import torch
    if stream is None:
        return None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {dev}")
    return torch.cuda.stream(stream)


def _need(dev, what, t, dtype, shape):
    """t is a contiguous tensor on dev of `dtype` and `shape`."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return
    if t.device != dev:
        raise ValueError(f"{what} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{what} must be contiguous")


def _cuda_device(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


def _dims(t, what, n):
    s = t.shape
    if len(s) != n:
        raise ValueError(f"{what} must have {n} dimensions, got {len(s)}")
    if t.numel() >= 2 ** 31 and max(s) >= 2 ** 31:
        raise ValueError(f"{what}: shape {tuple(s)}, a dimension does not fit 32 bits")
    return s


def _step(q_lat, q_rope, kv_cache, block_table, seq_lens, softmax_scale, causal, k_rope_cache, kv_scale, out_dtype,
          num_workers, kernel):
    """Checks that the tensors of a decode step fit one another; their device and parameters."""
    import torch
    dev = _cuda_device(q_lat, "q_lat")
    B, Sq, H, r = _dims(q_lat, "q_lat", 4)
    d_r = 0 if q_rope is None else _dims(q_rope, "q_rope", 4)[3]
    nb, bs, _ = _dims(kv_cache, "kv_cache", 3)
    mb = _dims(block_table, "block_table", 2)[1]
    ct = kv_cache.dtype
    cd = _dtype_code(kv_cache, "kv_cache")
    qt = torch.bfloat16 if cd == _b.E4M3 else ct
    _need(dev, "q_lat", q_lat, qt, (B, Sq, H, r))
    if q_rope is not None:
        _need(dev, "q_rope", q_rope, qt, (B, Sq, H, d_r))
    if cd == _b.E4M3:
        _need(dev, "kv_cache", kv_cache, ct, (nb, bs, r))
        if kv_scale is None or (d_r > 0 and k_rope_cache is None):
            raise ValueError("an e4m3 cache needs k_rope_cache and kv_scale")
        if k_rope_cache is not None:
            _need(dev, "k_rope_cache", k_rope_cache, torch.bfloat16, (nb, bs, d_r))
        _need(dev, "kv_scale", kv_scale, torch.float32, (nb, bs))
    else:
        _need(dev, "kv_cache", kv_cache, ct, (nb, bs, r + d_r))
        if k_rope_cache is not None or kv_scale is not None:
            raise ValueError("k_rope_cache and kv_scale belong to an e4m3 cache")
    _need(dev, "block_table", block_table, torch.int32, (B, mb))
    _need(dev, "seq_lens", seq_lens, torch.int32, (B,))
    qd = _b.BF16 if cd == _b.E4M3 else cd
    if out_dtype is None:
        out_dtype = qd
    return dev, _b.Params(B, Sq, H, r, d_r, bs, nb, mb, qd, cd, out_dtype, 1 if causal else 0, softmax_scale,
                          _b.int32(num_workers, "num_workers"), _b.KERNELS[kernel] if isinstance(kernel, str) else kernel, 0)


_workspace_bytes = {}   # (device, parameters) -> _window_workspace, a function of nothing else


def _window_workspace(p):
    """Bytes that a window decode of these parameters needs."""
    if p.cache_dtype == _b.E4M3 and p.kernel == _b.KERNELS["tc_pair"]:   # sized as the decode's own e4m3 kernel
        p = _b.Params.from_buffer_copy(p)
        p.kernel = _b.KERNELS["tcgen05"]
    return max(_b.workspace_size(p), 1)


def window_decode(q_lat, q_rope, kv_cache, block_table, seq_lens, softmax_scale, window, sinks=0, causal=False,
                  k_rope_cache=None, kv_scale=None, out=None, lse=None, workspace=None, out_dtype=None, num_workers=0,
                  kernel="auto", stream=None):
    """One MLA decode step over a sliding window and sink tokens (see mla_window_decode).

    A query row with n tokens (its own the last) sees tokens t < n with t >= n - window or t < sinks.
    Other arguments and the returned (out, lse) are decode's.
    """
    import torch
    dev, p = _step(q_lat, q_rope, kv_cache, block_table, seq_lens, softmax_scale, causal, k_rope_cache, kv_scale,
                   out_dtype, num_workers, kernel)
    away = _away(dev, stream)
    if away is not None:
        with away:
            return window_decode(q_lat, q_rope, kv_cache, block_table, seq_lens, softmax_scale, window, sinks, causal,
                                 k_rope_cache, kv_scale, out, lse, workspace, out_dtype, num_workers, kernel)
    shape = q_lat.shape
    B, Sq, H, _ = shape
    od = torch.float32 if p.out_dtype == _b.F32 else torch.bfloat16
    if out is None:
        out = torch.empty_like(q_lat, dtype=od)
    else:
        _need(dev, "out", out, od, shape)
    if lse is None:
        lse = torch.empty_strided((B, Sq, H), (Sq * H, H, 1), dtype=torch.float32, device=dev)
    else:
        _need(dev, "lse", lse, torch.float32, shape[:3])
    if workspace is None:
        key = (dev.index, bytes(p))
        n = _workspace_bytes.get(key)
        if n is None:
            if len(_workspace_bytes) >= 4096:
                _workspace_bytes.clear()
            n = _workspace_bytes[key] = _window_workspace(p)
        workspace = torch.empty_strided((n,), (1,), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of q_lat")
    _b.mla_window_decode(p, window, sinks, q_lat, q_rope, kv_cache, k_rope_cache, kv_scale, block_table, seq_lens, out, lse,
                         workspace, stream=_raw_stream(dev))
    return out, lse


def attention_mass(q_lat, q_rope, kv_cache, block_table, seq_lens, lse, softmax_scale, mass, mass_in=None,
                   causal=False, k_rope_cache=None, kv_scale=None, num_workers=0, kernel="auto", stream=None):
    """mass[b, t] = mass_in[b, t] + the attention weight that token t receives from all query rows
    of this step, for t < seq_lens[b] (see mla_attention_mass).

    lse [B, Sq, H] is the decode's over the whole cache (not window_decode's); mass float32 [B, max_seq_len]; mass_in of the same shape, or mass
    itself to add in place, or None for zeros. Entries past a sequence's length are left as they are.
    Returns mass.
    """
    import torch
    dev, p = _step(q_lat, q_rope, kv_cache, block_table, seq_lens, softmax_scale, causal, k_rope_cache, kv_scale, None,
                   num_workers, kernel)
    shape = q_lat.shape
    _need(dev, "lse", lse, torch.float32, shape[:3])
    S = _dims(mass, "mass", 2)[1]
    _need(dev, "mass", mass, torch.float32, (shape[0], S))
    if mass_in is not None and mass_in is not mass:
        _need(dev, "mass_in", mass_in, torch.float32, (shape[0], S))
    away = _away(dev, stream)
    if away is not None:
        with away:
            _b.mla_attention_mass(p, S, q_lat, q_rope, kv_cache, k_rope_cache, kv_scale, block_table, seq_lens, lse,
                                  mass_in, mass)
        return mass
    _b.mla_attention_mass(p, S, q_lat, q_rope, kv_cache, k_rope_cache, kv_scale, block_table, seq_lens, lse, mass_in, mass,
                          stream=_raw_stream(dev))
    return mass


def evict_select(mass, seq_lens, budget, sinks=0, recent=0, indices=None, counts=None, stream=None):
    """The tokens that stay when every sequence is cut to `budget`: the first `sinks`, the last `recent`
    and the heaviest between (see mla_evict_select). Returns (indices int32 [B, budget] ascending, -1
    padded; counts int32 [B]), the list that sparse_decode and cache_compact take."""
    import torch
    dev = _cuda_device(mass, "mass")
    B, S = _dims(mass, "mass", 2)
    i32 = torch.int32
    budget, sinks, recent = _b.int32(budget, "budget"), _b.int32(sinks, "sinks"), _b.int32(recent, "recent")
    _need(dev, "mass", mass, torch.float32, (B, S))
    _need(dev, "seq_lens", seq_lens, i32, (B,))
    if indices is not None:
        _need(dev, "indices", indices, i32, (B, budget))
    if counts is not None:
        _need(dev, "counts", counts, i32, (B,))
    away = _away(dev, stream)
    if away is not None:
        with away:
            return evict_select(mass, seq_lens, budget, sinks, recent, indices, counts)
    if indices is None:
        indices = torch.empty_strided((B, max(budget, 0)), (max(budget, 1), 1), dtype=i32, device=dev)
    if counts is None:
        counts = torch.empty_like(seq_lens)
    _b.mla_evict_select(_b.EvictParams(B, S, budget, sinks, recent, 0), mass, seq_lens, indices, counts,
                        stream=_raw_stream(dev))
    return indices, counts


def cache_compact(kv_cache, block_table, dst_block_table, indices, counts, k_rope_cache=None, kv_scale=None, mass=None,
                  mass_out=None, stream=None):
    """Copy the listed tokens into the (free) blocks of dst_block_table, in list order (see
    mla_cache_compact): counts are the sequences' lengths under the new table. With mass and mass_out
    (two buffers) the tokens' weights move along, and the rest of each mass_out row becomes 0. The RoPE keys
    stay rotated for the positions the tokens had: cache_append then takes rope=False and keys rotated for
    their places in the whole sequence. Returns None."""
    import torch
    dev = _cuda_device(kv_cache, "kv_cache")
    nb, bs, width = _dims(kv_cache, "kv_cache", 3)
    B, k = _dims(indices, "indices", 2)
    i32, f32 = torch.int32, torch.float32
    cd = _dtype_code(kv_cache, "kv_cache")
    mb, db = _dims(block_table, "block_table", 2)[1], _dims(dst_block_table, "dst_block_table", 2)[1]
    _need(dev, "kv_cache", kv_cache, kv_cache.dtype, (nb, bs, width))
    _need(dev, "block_table", block_table, i32, (B, mb))
    _need(dev, "dst_block_table", dst_block_table, i32, (B, db))
    _need(dev, "indices", indices, i32, (B, k))
    _need(dev, "counts", counts, i32, (B,))
    d_r = ms = mo = 0
    if k_rope_cache is not None:
        d_r = _dims(k_rope_cache, "k_rope_cache", 3)[2]
        _need(dev, "k_rope_cache", k_rope_cache, torch.bfloat16, (nb, bs, d_r))
    if kv_scale is not None:
        _need(dev, "kv_scale", kv_scale, f32, (nb, bs))
    if mass is not None:
        ms = _dims(mass, "mass", 2)[1]
        _need(dev, "mass", mass, f32, (B, ms))
    if mass_out is not None:
        mo = _dims(mass_out, "mass_out", 2)[1]
        _need(dev, "mass_out", mass_out, f32, (B, mo))
    p = _b.CompactParams(B, width, d_r, bs, nb, mb, db, cd, k, ms, mo, 0)
    away = _away(dev, stream)
    if away is not None:
        with away:
            _b.mla_cache_compact(p, kv_cache, k_rope_cache, kv_scale, block_table, dst_block_table, indices, counts, mass,
                                 mass_out)
        return
    _b.mla_cache_compact(p, kv_cache, k_rope_cache, kv_scale, block_table, dst_block_table, indices, counts, mass, mass_out,
                         stream=_raw_stream(dev))


def verify_drafts(target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens=None, seq_lens=None,
                  tokens=None, accepted=None, new_seq_lens=None, stream=None):
    """Accept the longest prefix of the drafted tokens that the target's probabilities allow, and draw one
    more token (see mla_verify_drafts).

    target_probs [B, K + 1, V] and draft_probs [B, K, V] (or None: the drafts were not sampled), both
    float32 or both bfloat16; draft_tokens int32 [B, K]; accept_u float32 [B, K] and sample_u float32
    [B] uniform in [0, 1); draft_lens int32 [B] when sequences have fewer than K drafts. Returns (tokens
    int32 [B, K + 1], -1 padded, accepted int32 [B]), and with seq_lens (the cache's lengths, drafts
    included) also new_seq_lens int32 [B] without the refused drafts.
    """
    import torch
    dev = _cuda_device(target_probs, "target_probs")
    B, K1, V = _dims(target_probs, "target_probs", 3)
    K = K1 - 1
    pt, i32 = target_probs.dtype, torch.int32
    pd = _b.F32 if pt is torch.float32 else _b.BF16
    _need(dev, "target_probs", target_probs, pt if pt is torch.float32 else torch.bfloat16, (B, K1, V))
    if draft_probs is not None:
        _need(dev, "draft_probs", draft_probs, pt, (B, K, V))
    _need(dev, "draft_tokens", draft_tokens, i32, (B, K))
    _need(dev, "accept_u", accept_u, torch.float32, (B, K))
    _need(dev, "sample_u", sample_u, torch.float32, (B,))
    if draft_lens is not None:
        _need(dev, "draft_lens", draft_lens, i32, (B,))
    if seq_lens is not None:
        _need(dev, "seq_lens", seq_lens, i32, (B,))
    elif new_seq_lens is not None:
        raise ValueError("new_seq_lens needs seq_lens")
    if tokens is not None:
        _need(dev, "tokens", tokens, i32, (B, K1))
    if accepted is not None:
        _need(dev, "accepted", accepted, i32, (B,))
    if new_seq_lens is not None:
        _need(dev, "new_seq_lens", new_seq_lens, i32, (B,))
    away = _away(dev, stream)
    if away is not None:
        with away:
            return verify_drafts(target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens, seq_lens, tokens,
                                 accepted, new_seq_lens)
    if tokens is None:
        tokens = torch.empty_strided((B, K1), (K1, 1), dtype=i32, device=dev)
    if accepted is None:
        accepted = torch.empty_strided((B,), (1,), dtype=i32, device=dev)
    if seq_lens is not None and new_seq_lens is None:
        new_seq_lens = torch.empty_like(seq_lens)
    _b.mla_verify_drafts(_b.VerifyParams(B, K, V, pd, 0), target_probs, draft_probs, draft_tokens, draft_lens, accept_u,
                         sample_u, seq_lens, tokens, accepted, new_seq_lens, stream=_raw_stream(dev))
    return (tokens, accepted) if seq_lens is None else (tokens, accepted, new_seq_lens)
