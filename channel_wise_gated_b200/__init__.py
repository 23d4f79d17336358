"""Kimi Delta Attention (KDA) on B200: chunkwise prefill and recurrent decode.

Thin Python binding over the C ABI of ``include/kda.h``. PyTorch is used only to
hold device memory and to name the current CUDA stream; every step of the
operator runs in the library's CUDA kernels. Functions take torch tensors,
check their dtypes, shapes and contiguity, and pass raw pointers through.

    o, hT = chunk_fwd(q, k, v, log_alpha, beta, h0=None, cu_seqlens=None)
    o     = decode_step(q, k, v, log_alpha, beta, state)      # state updated in place
    o     = decode_tokens(q, k, v, log_alpha, beta, state)    # t tokens per sequence
    o     = decode_tree(q, k, v, log_alpha, beta, state, tree)  # a tree of drafted tokens

The latent-attention (MLA) layers that alternate with KDA layers, over a paged cache:

    mla_append(x, norm_w, cache, page_table, cache_lens, cu_seqlens)
    o, lse = mla_prefill(q, k, k_shared, v, cu_seqlens)               # expanded form
    o, lse = mla_decode(q, cache, page_table, cache_lens, tree=None)  # absorbed form
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _native
from ._native import KdaError  # noqa: F401

D = 128
MLA_LATENT = 512                        # latent values per token, shared by all heads
MLA_SHARED = 64                         # key values per token that the heads share as they are
MLA_WIDTH = MLA_LATENT + MLA_SHARED     # values cached per token

# Arithmetic type of the prefill contractions for bf16 inputs (bf16 operands, fp32 accumulation).
PREFILL_COMPUTE_DTYPE = "bf16"

_DT = {torch.float32: _native.KDA_F32, torch.bfloat16: _native.KDA_BF16}


def _need(t: torch.Tensor, name: str, dtype=None, shape=None, device=None):
    if (shape is not None and device is not None and isinstance(t, torch.Tensor) and t.is_cuda
            and t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return   # (all is well in one pass; what is not is named below)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(fn, dev, *args) -> int:
    """Call an entry point on dev's current stream, with dev the current device; its status. (A
    device guard and a Stream object cost 3.6 us of a call's host time: the guard is taken only
    where it is needed, the stream's handle read as it is.)"""
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch.cuda.current_device() == dev.index:
        return fn(*args, stream)
    with torch.cuda.device(dev):
        return fn(*args, stream)


def _launch(fn, where, dev, *args):
    """_call, with a status other than KDA_OK raised."""
    st = _call(fn, dev, *args)
    if st:
        _native.check(st, where)


def _prefill_args(q, k, v, gate, gate_shape_tail, beta, h0, cu_seqlens, o, hT,
                  output_final_state, check_gate=True):
    """Check a prefill call's tensors and allocate missing outputs; returns the
    pointer tuple of the C prefill entry points and (o, hT, N, T, H)."""
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must be [T, H, 128]")
    T, H, _ = q.shape
    dev = q.device
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, (T, H, D), dev)
    if check_gate:
        _need(gate, "log gate", torch.float32, (T, H) + gate_shape_tail, dev)
    _need(beta, "beta", torch.float32, (T, H), dev)
    if cu_seqlens is None:
        N = 1
    else:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [N+1]")
        N = cu_seqlens.numel() - 1
    if h0 is not None:
        _need(h0, "h0", torch.float32, (N, H, D, D), dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, (T, H, D), dev)
    if output_final_state and hT is None:
        hT = torch.empty((N, H, D, D), dtype=torch.float32, device=dev)
    elif hT is not None:
        _need(hT, "hT", torch.float32, (N, H, D, D), dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
            N, T, H, _DT[q.dtype], _ptr(o), _ptr(hT))
    return args, (o, hT, N, T, H)


def dplr_chunk_fwd(q, k, v, a, b, log_alpha, h0=None, cu_seqlens=None, o=None, hT=None,
                   output_final_state: bool = True):
    """General DPLR prefill (comparison kernel): S_t = (Diag(alpha_t) - a_t b_t^T) S_{t-1} +
    k_t v_t^T. q, k, v, a, b: [T, H, 128] bf16 or fp32 (same dtype); log_alpha: [T, H, 128]
    fp32; h0, cu_seqlens as chunk_fwd. Returns (o, hT)."""
    lib = _native.load()
    for name, t in (("a", a), ("b", b)):
        _need(t, name, q.dtype, tuple(q.shape), q.device)
    T, H, _ = q.shape
    dummy_beta = torch.empty((T, H), dtype=torch.float32, device=q.device)
    args, (o, hT, N, T, H) = _prefill_args(q, k, v, log_alpha, (D,), dummy_beta, h0, cu_seqlens,
                                           o, hT, output_final_state)
    q_, k_, v_, la_, _, h0_, cu_, N_, T_, H_, dt_, o_, hT_ = args
    _launch(lib.kda_dplr_chunk_fwd, "kda_dplr_chunk_fwd", q.device, q_, k_, v_, _ptr(a), _ptr(b),
            la_, h0_, cu_, N_, T_, H_, dt_, o_, hT_)
    return o, hT


def short_conv_swish(x, w, cu_seqlens=None, y=None):
    """Causal 4-tap depthwise convolution + Swish over tokens, restarted per sequence.

    x: [T, H, 128] (or [T, C]) bf16; w: [C, 4] fp32 with C = H * 128; cu_seqlens:
    [N+1] int32 on the device or None. Returns y like x.
    """
    lib = _native.load()
    dev = x.device
    T = x.shape[0]
    C = x.numel() // max(T, 1) if T else int(torch.tensor(x.shape[1:]).prod())
    _need(x, "x", torch.bfloat16, None, dev)
    _need(w, "w", torch.float32, (C, 4), dev)
    if cu_seqlens is None:
        N = 1
    else:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        N = cu_seqlens.numel() - 1
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", torch.bfloat16, tuple(x.shape), dev)
    _launch(lib.kda_short_conv_swish, "kda_short_conv_swish", dev, _ptr(x), _ptr(w),
            _ptr(cu_seqlens), N, T, C, _ptr(y))
    return y


def chunk_fwd_fused(q_pre, k_pre, v, decay_pre, beta_pre, gate_pre, norm_w, h0=None,
                    cu_seqlens=None, o=None, hT=None, output_final_state: bool = True,
                    split: bool = True):
    """KDA prefill with the layer's activations and output gate fused in.

    q_pre, k_pre, v, decay_pre, gate_pre: [T, H, 128] bf16; beta_pre: [T, H] fp32;
    norm_w: [128] fp32. q and k are L2-normalised in the kernel, log alpha =
    logsigmoid(decay_pre), beta = sigmoid(beta_pre), and the output is the head-wise
    RMSNorm of o times norm_w times sigmoid(gate_pre). Returns (o_out, hT).
    """
    lib = _native.load()
    T, H, _ = q_pre.shape
    dev = q_pre.device
    _need(q_pre, "q_pre", torch.bfloat16, (T, H, D), dev)
    _need(decay_pre, "decay_pre", torch.bfloat16, (T, H, D), dev)
    _need(gate_pre, "gate_pre", torch.bfloat16, (T, H, D), dev)
    _need(norm_w, "norm_w", torch.float32, (D,), dev)
    args, (o, hT, N, T, H) = _prefill_args(q_pre, k_pre, v, None, None, beta_pre, h0,
                                           cu_seqlens, o, hT, output_final_state,
                                           check_gate=False)
    ws_bytes = 0
    if split:
        ws_bytes = lib.kda_chunk_fwd_workspace_size(N, T, H, _native.KDA_BF16,
                                                    int(cu_seqlens is not None))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    q_, k_, v_, _, b_, h0_, cu_, N_, T_, H_, _, o_, hT_ = args
    _launch(lib.kda_chunk_fwd_fused, "kda_chunk_fwd_fused", dev, q_, k_, v_, _ptr(decay_pre), b_,
            _ptr(gate_pre), _ptr(norm_w), h0_, cu_, N_, T_, H_, o_, hT_, _ptr(ws), ws_bytes)
    return o, hT


def gdn_chunk_fwd(q, k, v, log_a, beta, h0=None, cu_seqlens=None, o=None, hT=None,
                  output_final_state: bool = True, split: bool = True):
    """Chunkwise Gated DeltaNet prefill: KDA with one scalar gate per token and head.

    q, k, v: [T, H, 128] bf16 or fp32; log_a: [T, H] fp32 (log of the gate);
    beta: [T, H] fp32; h0, cu_seqlens, o, hT: as chunk_fwd. With ``split`` a single
    long bf16 sequence is split in time over a workspace allocated here.
    """
    lib = _native.load()
    args, (o, hT, N, T, H) = _prefill_args(q, k, v, log_a, (), beta, h0, cu_seqlens, o, hT,
                                           output_final_state)
    ws_bytes = 0
    if split:
        ws_bytes = lib.kda_chunk_fwd_workspace_size(N, T, H, _DT[q.dtype],
                                                    int(cu_seqlens is not None))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _launch(lib.kda_gdn_chunk_fwd_ws, "kda_gdn_chunk_fwd_ws", q.device, *args, _ptr(ws), ws_bytes)
    return o, hT


def chunk_fwd(q, k, v, log_alpha, beta, h0=None, cu_seqlens=None, o=None, hT=None,
              output_final_state: bool = True, kernel: str = "auto"):
    """Chunkwise KDA prefill.

    q, k, v: [T, H, 128] bf16 or fp32 (same dtype); log_alpha: [T, H, 128] fp32;
    beta: [T, H] fp32; h0: [N, H, 128, 128] fp32 or None; cu_seqlens: [N+1] int32
    on the device or None (one sequence). Returns (o, hT) with o like q and hT
    [N, H, 128, 128] fp32 (None if output_final_state is False).
    ``kernel``: "auto" (tensor cores for bf16, CUDA cores for fp32; a single long
    bf16 sequence is split in time over a workspace allocated here), "static" (as
    "auto", with the library's module-resident scratch instead: no allocation),
    "single" (as "auto" but never split) or "simt" (always the fp32 CUDA-core chunk
    kernel).
    """
    lib = _native.load()
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must be [T, H, 128]")
    T, H, _ = q.shape
    dev = q.device
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, (T, H, D), dev)
    _need(log_alpha, "log_alpha", torch.float32, (T, H, D), dev)
    _need(beta, "beta", torch.float32, (T, H), dev)
    if cu_seqlens is None:
        N = 1
    else:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [N+1]")
        N = cu_seqlens.numel() - 1
    if h0 is not None:
        _need(h0, "h0", torch.float32, (N, H, D, D), dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, (T, H, D), dev)
    if output_final_state and hT is None:
        hT = torch.empty((N, H, D, D), dtype=torch.float32, device=dev)
    elif hT is not None:
        _need(hT, "hT", torch.float32, (N, H, D, D), dev)
    if kernel not in ("auto", "static", "single", "simt"):
        raise ValueError("kernel must be 'auto', 'static', 'single' or 'simt'")
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
            N, T, H, _DT[q.dtype], _ptr(o), _ptr(hT))
    if kernel == "simt":
        _launch(lib.kda_chunk_fwd_simt, "kda_chunk_fwd_simt", dev, *args)
    elif kernel == "static":
        _launch(lib.kda_chunk_fwd_static, "kda_chunk_fwd_static", dev, *args)
    else:
        ws_bytes = 0
        if kernel == "auto":
            ws_bytes = lib.kda_chunk_fwd_workspace_size(N, T, H, _DT[q.dtype],
                                                        int(cu_seqlens is not None))
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
        _launch(lib.kda_chunk_fwd_ws, "kda_chunk_fwd_ws", dev, *args, _ptr(ws), ws_bytes)
        # (the caching allocator keeps ws alive for the stream's use of it)
    return o, hT


def split_plan(n_heads: int, t_total: int, n_sms: int = 0, workspace_bytes: Optional[int] = None):
    """Segment bounds of the time split that kda_chunk_fwd_ws uses for one bf16
    sequence (token offsets, n + 1 of them), or [] when the single pass runs.
    n_sms = 0 plans for the current device; workspace_bytes None = unlimited."""
    import ctypes
    lib = _native.load()
    bounds = (ctypes.c_int64 * (_native.KDA_MAX_SEGMENTS + 1))()
    ws = _native.SIZE_MAX if workspace_bytes is None else int(workspace_bytes)
    n = lib.kda_chunk_fwd_split_plan(int(n_heads), int(t_total), int(n_sms), ws, bounds)
    if n < 0:
        raise KdaError(n, "kda_chunk_fwd_split_plan")
    return [int(bounds[i]) for i in range(n + 1)] if n >= 2 else []


def decode_step(q, k, v, log_alpha, beta, state, o=None):
    """One recurrent KDA step per (sequence, head), state updated in place.

    q, k, v: [N, H, 128] bf16 or fp32; log_alpha: [N, H, 128], beta: [N, H]
    (bf16 or fp32, same dtype); state: [N, H, 128, 128] fp32. Returns o like q.
    """
    lib = _native.load()
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must be [N, H, 128]")
    N, H, _ = q.shape
    dev = q.device
    if q.dtype not in _DT or log_alpha.dtype not in _DT:
        raise TypeError("unsupported dtype")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, (N, H, D), dev)
    _need(log_alpha, "log_alpha", log_alpha.dtype, (N, H, D), dev)
    _need(beta, "beta", log_alpha.dtype, (N, H), dev)
    _need(state, "state", torch.float32, (N, H, D, D), dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, (N, H, D), dev)
    _launch(lib.kda_decode_step, "kda_decode_step", dev, _ptr(q), _ptr(k), _ptr(v),
            _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(o), N, H, _DT[q.dtype],
            _DT[log_alpha.dtype])
    return o


def decode_tokens(q, k, v, log_alpha, beta, state, o=None):
    """Several recurrent KDA steps per (sequence, head) in one call, state in place.

    q, k, v: [N, t, H, 128] bf16 or fp32 (sequence-major, t = 1..16 new tokens per
    sequence); log_alpha: [N, t, H, 128] and beta: [N, t, H] (bf16 or fp32, same
    dtype); state: [N, H, 128, 128] fp32, read once and written once. Returns o like q.
    """
    lib = _native.load()
    if q.dim() != 4 or q.shape[3] != D:
        raise ValueError("q must be [N, t, H, 128]")
    N, t, H, _ = q.shape
    if not 1 <= t <= _native.KDA_DECODE_MAX_TOKENS:
        raise ValueError(f"t must be in 1..{_native.KDA_DECODE_MAX_TOKENS}")
    dev = q.device
    if q.dtype not in _DT or log_alpha.dtype not in _DT:
        raise TypeError("unsupported dtype")
    for name, x in (("q", q), ("k", k), ("v", v)):
        _need(x, name, q.dtype, (N, t, H, D), dev)
    _need(log_alpha, "log_alpha", log_alpha.dtype, (N, t, H, D), dev)
    _need(beta, "beta", log_alpha.dtype, (N, t, H), dev)
    _need(state, "state", torch.float32, (N, H, D, D), dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, (N, t, H, D), dev)
    _launch(lib.kda_decode_tokens, "kda_decode_tokens", dev, _ptr(q), _ptr(k), _ptr(v),
            _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(o), N, t, H, _DT[q.dtype],
            _DT[log_alpha.dtype])
    return o


def decode_tree(q, k, v, log_alpha, beta, state, tree=None, o=None):
    """Outputs of a tree of drafted tokens per (sequence, head); the state is only read.

    q, k, v: [N, t, H, 128] bf16 or fp32, t = 1..16; log_alpha: [N, t, H, 128] and beta:
    [N, t, H] (bf16 or fp32, same dtype); state: [N, H, 128, 128] fp32; tree: [N, t] int32,
    bit i of tree[n, r] set if token i is an ancestor of token r or r itself, parents before
    their children (None: a chain). Token r's output is the recurrence's after the tokens of
    its path. With bf16 q, k, v the products with the state are taken in two bf16 parts of each
    factor, off by at most 3 * 2^-16 of their terms' absolute sum; fp32 ones keep fp32's
    accuracy. Returns o like q. The accepted path is then applied with decode_tokens.
    """
    lib = _native.load()
    if q.dim() != 4 or q.shape[3] != D:
        raise ValueError("q must be [N, t, H, 128]")
    N, t, H, _ = q.shape
    if not 1 <= t <= _native.KDA_DECODE_MAX_TOKENS:
        raise ValueError(f"t must be in 1..{_native.KDA_DECODE_MAX_TOKENS}")
    dev = q.device
    if q.dtype not in _DT or log_alpha.dtype not in _DT:
        raise TypeError("unsupported dtype")
    for name, x in (("q", q), ("k", k), ("v", v)):
        _need(x, name, q.dtype, (N, t, H, D), dev)
    _need(log_alpha, "log_alpha", log_alpha.dtype, (N, t, H, D), dev)
    _need(beta, "beta", log_alpha.dtype, (N, t, H), dev)
    _need(state, "state", torch.float32, (N, H, D, D), dev)
    if tree is not None:
        _need(tree, "tree", torch.int32, (N, t), dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, (N, t, H, D), dev)
    _launch(lib.kda_decode_tree, "kda_decode_tree", dev, _ptr(q), _ptr(k), _ptr(v),
            _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(tree), _ptr(o), N, t, H, _DT[q.dtype],
            _DT[log_alpha.dtype])
    return o


def _rows(t, name, dtype, shape, device):
    """Check a tensor whose last dimension alone must be dense; returns its pointer and the other
    dimensions' strides, which are passed on (multiples of 8 elements, 16 bytes of bf16; of a
    dimension of one entry, where torch may report any, the dense one)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.shape == shape
            and (device is None or t.device == device)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if device is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    strides = t.stride()
    dense, odd, out = shape[-1], strides[-1] != 1, []
    for n, s in zip(shape[-2::-1], strides[-2::-1]):
        if n <= 1:
            s = dense
        odd = odd or s % 8
        out.append(s)
        dense = n * s
    if odd:
        raise ValueError(f"{name} must have a dense last dimension and strides in multiples of 8")
    return (t.data_ptr(), *out[::-1])


def _paged_cache(cache, page_table, cache_lens, n_seqs, dev):
    """Check a paged latent cache; returns (n_pages, page_size, max_pages)."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3 or cache.shape[2] != MLA_WIDTH:
        raise ValueError("cache must be [n_pages, page_size, 576]")
    _need(cache, "cache", torch.bfloat16, None, dev)
    _need(page_table, "page_table", torch.int32, None, dev)
    if page_table.dim() != 2 or page_table.shape[0] != n_seqs:
        raise ValueError(f"page_table must be [{n_seqs}, max_pages]")
    _need(cache_lens, "cache_lens", torch.int32, (n_seqs,), dev)
    return cache.shape[0], cache.shape[1], page_table.shape[1]


def mla_append(x, norm_w, cache, page_table, cache_lens, cu_seqlens=None, latent=None,
               output_latent: bool = False, eps: float = 1e-6):
    """Normalise new tokens' latents and write them into the paged cache (in place).

    x: [T, 576] bf16, 512 latent values and the 64 shared key values (rows may be strided, as
    a slice of a wider projection); norm_w: [512] fp32 RMSNorm weight or None (cached as they
    are); cache: [n_pages, page_size, 576] bf16; page_table: [N, max_pages] int32; cache_lens:
    [N] int32, lengths with the new tokens: sequence n's T_n new rows are the last ones before
    cache_lens[n]; cu_seqlens: [N+1] int32 or None (T / N tokens each). Returns the normalised
    latents [T, 512] bf16 with output_latent (or into latent), else None.
    """
    lib = _native.load()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [T, 576]")
    dev, T = x.device, x.shape[0]
    xs = _rows(x, "x", torch.bfloat16, (T, MLA_WIDTH), None)
    _need(cache_lens, "cache_lens", torch.int32, None, dev)
    N = cache_lens.numel()
    n_pages, page_size, max_pages = _paged_cache(cache, page_table, cache_lens, N, dev)
    if norm_w is not None:
        _need(norm_w, "norm_w", torch.float32, (MLA_LATENT,), dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    if latent is not None:
        _need(latent, "latent", torch.bfloat16, (T, MLA_LATENT), dev)
    elif output_latent:
        latent = torch.empty((T, MLA_LATENT), dtype=torch.bfloat16, device=dev)
    _launch(lib.kda_mla_append, "kda_mla_append", dev, *xs, _ptr(norm_w), float(eps), _ptr(cache),
            n_pages, page_size, _ptr(page_table), max_pages, _ptr(cache_lens), _ptr(cu_seqlens), N,
            T, _ptr(latent))
    return latent


def mla_prefill(q, k, k_shared, v, cu_seqlens=None, cu_seqlens_k=None, scale=None,
                causal: bool = True, o=None, lse=None, output_lse: bool = False):
    """Latent attention, expanded form: softmax attention of a packed batch.

    q: [Tq, H, 192]; k, v: [Tk, H, 128] (expanded from the latents); k_shared: [Tk, 64], the
    heads' shared key values, against q's last 64; all bf16, strided views allowed with a dense
    last dimension. cu_seqlens: [N+1] int32 or None (one sequence); cu_seqlens_k: the keys'
    where they differ (a prefix cached before): with causal a sequence's last query sees its
    last key. scale: 1 / sqrt(192) by default. Returns (o, lse): o [Tq, H, 128] bf16, lse
    [Tq, H] fp32 with output_lse (or into lse), else None.
    """
    lib = _native.load()
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [Tq, H, 192]")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be [Tk, H, 128]")
    dev, (Tq, H, _), Tk = q.device, q.shape, k.shape[0]
    qs = _rows(q, "q", torch.bfloat16, (Tq, H, D + MLA_SHARED), None)
    k_ = _rows(k, "k", torch.bfloat16, (Tk, H, D), dev)
    vs = _rows(v, "v", torch.bfloat16, (Tk, H, D), dev)
    shs = _rows(k_shared, "k_shared", torch.bfloat16, (Tk, MLA_SHARED), dev)
    N = 1
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [N+1]")
        N = cu_seqlens.numel() - 1
        if cu_seqlens_k is not None:
            _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, (N + 1,), dev)
        elif Tk != Tq:
            raise ValueError("cu_seqlens_k is needed where queries and keys differ in number")
        else:
            cu_seqlens_k = cu_seqlens
    elif cu_seqlens_k is not None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    if o is None:
        o = q.new_empty((Tq, H, D))
    else:
        _need(o, "o", torch.bfloat16, (Tq, H, D), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (Tq, H), dev)
    elif output_lse:
        lse = q.new_empty((Tq, H), dtype=torch.float32)
    if scale is None:
        scale = (D + MLA_SHARED) ** -0.5

    _launch(lib.kda_mla_prefill, "kda_mla_prefill", dev, *qs, *k_, *shs, *vs, _ptr(cu_seqlens),
            _ptr(cu_seqlens_k), N, Tq, Tk, H, float(scale), int(causal), _ptr(o), _ptr(lse))
    return o, lse


def mla_decode_workspace_size(n_tokens: int, n_heads: int, device=None) -> int:
    """Bytes of workspace that mla_decode takes on the device (default: the current one), for any
    number and length of sequences."""
    lib = _native.load()
    dev = None if device is None else torch.device(device).index
    if dev is None or dev == torch.cuda.current_device():
        return lib.kda_mla_decode_workspace_size(int(n_tokens), int(n_heads))
    with torch.cuda.device(dev):
        return lib.kda_mla_decode_workspace_size(int(n_tokens), int(n_heads))


def mla_decode(q, cache, page_table, cache_lens, tree=None, scale=None, o=None, lse=None,
               output_lse: bool = False, workspace=None):
    """Latent attention, absorbed form: 1 to 16 new tokens per sequence over the paged cache.

    q: [N, t, H, 576] bf16 (queries multiplied into the latent space, then their 64 shared
    values); cache: [n_pages, page_size, 576] bf16, page_size a multiple of 8; page_table: [N,
    max_pages] int32; cache_lens: [N] int32, lengths with the t new tokens, which mla_append has
    written; tree: [N, t] int32 ancestor bits as decode_tree, or None (a chain). scale:
    1 / sqrt(192) by default. workspace: uint8 of mla_decode_workspace_size bytes, allocated
    here if None; calls that may overlap need one each. Returns (o, lse): o [N, t, H, 512] bf16
    in the latent space, lse [N, t, H] fp32 with output_lse (or into lse), else None.
    """
    lib = _native.load()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != MLA_WIDTH:
        raise ValueError("q must be [N, t, H, 576]")
    N, t, H, _ = q.shape
    if not 1 <= t <= _native.KDA_DECODE_MAX_TOKENS:
        raise ValueError(f"t must be in 1..{_native.KDA_DECODE_MAX_TOKENS}")
    _need(q, "q", torch.bfloat16)
    dev = q.device
    n_pages, page_size, max_pages = _paged_cache(cache, page_table, cache_lens, N, dev)
    if page_size % 8:
        raise ValueError("page_size must be a multiple of 8")
    if tree is not None:
        _need(tree, "tree", torch.int32, (N, t), dev)
    if o is None:
        o = q.new_empty((N, t, H, MLA_LATENT))
    else:
        _need(o, "o", torch.bfloat16, (N, t, H, MLA_LATENT), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (N, t, H), dev)
    elif output_lse:
        lse = q.new_empty((N, t, H), dtype=torch.float32)
    if scale is None:
        scale = (D + MLA_SHARED) ** -0.5
    if workspace is None:
        workspace = q.new_empty(mla_decode_workspace_size(t, H, dev), dtype=torch.uint8)
    else:
        _need(workspace, "workspace", torch.uint8, None, dev)
    _launch(lib.kda_mla_decode, "kda_mla_decode", dev, _ptr(q), _ptr(cache), n_pages, page_size,
            _ptr(page_table), max_pages, _ptr(cache_lens), _ptr(tree), N, t, H, float(scale),
            _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel())
    return o, lse


def device_status(device=None) -> int:
    """Read and clear the library's error word on the device (default: the current one);
    synchronises that device's current stream."""
    lib = _native.load()
    dev = torch.device("cuda") if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return int(_call(lib.kda_device_status, dev))
