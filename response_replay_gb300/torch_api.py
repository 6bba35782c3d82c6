"""PyTorch-facing helpers over the C ABI.

PyTorch supplies device memory and streams; every step of the computation runs in the
CUDA kernels behind include/longstraw.h.  These helpers allocate outputs and workspace
with torch, check shapes and dtypes, and pass raw pointers to the binding.
"""
from __future__ import annotations

import threading

import torch

from . import binding as B

HEAD_DIM = 128


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(t: torch.Tensor, name: str, dtype, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


_workspaces: dict = {}


class _StreamWorkspace:
    """The workspace of the calls of one kind on one stream, and the lock of its users."""

    __slots__ = ("lock", "buf")

    def __init__(self):
        self.lock, self.buf = threading.RLock(), None  # a finalizer may call


_stream_workspaces: dict = {}
_captured_workspaces: list = []  # of captures that torch does not know of


def _graph_memory(t: torch.Tensor) -> bool:
    """Whether t, made during a capture, lies in memory that is the graph's: in a pool of its
    own (that of the torch.cuda.CUDAGraph being captured), not in the one that all tensors
    share; or from the stream-ordered allocator, whose allocations and releases are captured
    themselves.  An allocator that does not say counts as shared."""
    if torch.cuda.get_allocator_backend() == "cudaMallocAsync":
        return True
    try:
        segments = torch.cuda.memory_snapshot()
    except RuntimeError:
        return False
    p = t.data_ptr()
    return any(s["address"] <= p < s["address"] + s["total_size"] and tuple(s["segment_pool_id"]) != (0, 0)
               for s in segments)


def _with_workspace(call, args: tuple, size, like: torch.Tensor, key: str, stream: int) -> None:
    """call(*args, workspace, its bytes, stream) with the workspace of the calls of one kind
    on the current stream (calls on different streams may overlap).  A call launches kernels
    that talk through it, and other host threads run while it does, so it holds the
    workspace's lock: two threads' calls on one stream go in whole, one behind the other.  It
    grows when the call says that it is too small, which it does before it launches anything.
    A captured call takes one of its own (two graphs captured on one stream may be replayed
    on two): from the graph's memory, or, in a capture that torch does not make, from all
    tensors' memory, where it stays taken as long as the process lives, as nothing says when
    such a graph's last replay has been."""
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(max(size(), 256), dtype=torch.uint8, device=like.device)
        if not _graph_memory(ws):
            _captured_workspaces.append(ws)
        return call(*args, ws.data_ptr(), ws.numel(), stream)
    k = (like.get_device(), key, stream)
    entry = _stream_workspaces.get(k)
    if entry is None:
        entry = _stream_workspaces.setdefault(k, _StreamWorkspace())
    with entry.lock:
        ws = entry.buf
        if ws is not None:
            try:
                return call(*args, ws.data_ptr(), ws.numel(), stream)
            except B.LongstrawError as e:
                if e.status != B.LS_ERR_WORKSPACE:
                    raise
        entry.buf = ws = torch.empty(max(size(), 256), dtype=torch.uint8, device=like.device)
        call(*args, ws.data_ptr(), ws.numel(), stream)


def workspace(nbytes: int, device: torch.device, key: str = "default") -> torch.Tensor:
    """A reusable uint8 workspace of at least nbytes on `device` (grown on demand).
    Calls that share a key must not overlap on the GPU."""
    k = (device.index if device.index is not None else torch.cuda.current_device(), key)
    ws = _workspaces.get(k)
    if ws is None or ws.numel() < max(nbytes, 1):
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[k] = ws
    return ws


def _check_pool(t: torch.Tensor, name: str, shape):
    """A page pool: GPU memory, or pinned host memory the GPU reads directly."""
    if not t.is_cuda and not (t.device.type == "cpu" and t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or a pinned host tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


class PagedKVCache:
    """K/V page pools plus page table of one attention layer (ls_kv_cache).

    host_pools=True places the pools in pinned host memory (on a Grace-Blackwell node,
    Grace memory read over NVLink-C2C); the kernels read and write them there."""

    def __init__(self, num_pages: int, page_table: torch.Tensor, page_size: int, num_kv_heads: int,
                 num_tokens: int, device=None, fill: float | None = None,
                 k_pool: torch.Tensor | None = None, v_pool: torch.Tensor | None = None,
                 host_pools: bool = False):
        device = torch.device(device) if device is not None else page_table.device
        shape = (num_pages, num_kv_heads, page_size, HEAD_DIM)
        if k_pool is None:
            if host_pools:
                k_pool = torch.empty(shape, dtype=torch.bfloat16, pin_memory=True)
                v_pool = torch.empty(shape, dtype=torch.bfloat16, pin_memory=True)
            else:
                k_pool = torch.empty(shape, dtype=torch.bfloat16, device=device)
                v_pool = torch.empty(shape, dtype=torch.bfloat16, device=device)
            if fill is not None:
                k_pool.fill_(fill)
                v_pool.fill_(fill)
        _check_pool(k_pool, "k_pool", shape)
        _check_pool(v_pool, "v_pool", shape)
        _check(page_table, "page_table", torch.int32)
        self.k_pool, self.v_pool, self.page_table = k_pool, v_pool, page_table
        self.page_size, self.num_kv_heads, self.num_tokens = page_size, num_kv_heads, num_tokens
        self.struct = B.ls_kv_cache(k_pool.data_ptr(), v_pool.data_ptr(), page_table.data_ptr(),
                                    num_pages, page_table.numel(), page_size, num_kv_heads,
                                    HEAD_DIM, num_tokens)

    @property
    def device(self):
        return self.page_table.device

    def capture(self, k: torch.Tensor, v: torch.Tensor, start_pos: int = 0, stream=None) -> None:
        n = k.shape[0]
        _check(k, "k", torch.bfloat16, (n, self.num_kv_heads, HEAD_DIM))
        _check(v, "v", torch.bfloat16, (n, self.num_kv_heads, HEAD_DIM))
        B.ls_capture_kv(self.struct, k.data_ptr(), v.data_ptr(), start_pos, n, _stream(stream))

    def validate(self, stream=None) -> None:
        nbytes = B.ls_validate_page_table_workspace(self.struct)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        B.ls_validate_page_table(self.struct, ws.data_ptr(), nbytes, _stream(stream))


def replay_fwd(cache: PagedKVCache, q: torch.Tensor, k_resp: torch.Tensor, v_resp: torch.Tensor,
               softmax_scale: float, num_splits: int, o: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, stream=None):
    R, hq, _ = q.shape
    _check(q, "q", torch.bfloat16, (R, hq, HEAD_DIM))
    _check(k_resp, "k_resp", torch.bfloat16, (R, cache.num_kv_heads, HEAD_DIM))
    _check(v_resp, "v_resp", torch.bfloat16, (R, cache.num_kv_heads, HEAD_DIM))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((R, hq), dtype=torch.float32, device=q.device)
    _check(o, "o", torch.bfloat16, q.shape)
    _check(lse, "lse", torch.float32, (R, hq))
    nbytes = B.ls_replay_attn_fwd_workspace(cache.struct, R, hq, num_splits)
    ws = workspace(nbytes, q.device, "fwd")
    B.ls_replay_attn_fwd(cache.struct, q.data_ptr(), k_resp.data_ptr(), v_resp.data_ptr(), R, hq,
                         softmax_scale, num_splits, o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                         ws.numel(), _stream(stream))
    return o, lse


def replay_fwd_members(cache: PagedKVCache, q: torch.Tensor, k_resp: torch.Tensor,
                       v_resp: torch.Tensor, softmax_scale: float, num_splits: int,
                       o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       stream=None):
    """Forward of several equal-length responses over the prompt in one launch:
    q [members][R][Hq][128], k_resp / v_resp [members][R][Hkv][128]."""
    M, R, hq, _ = q.shape
    hkv = cache.num_kv_heads
    _check(q, "q", torch.bfloat16, (M, R, hq, HEAD_DIM))
    _check(k_resp, "k_resp", torch.bfloat16, (M, R, hkv, HEAD_DIM))
    _check(v_resp, "v_resp", torch.bfloat16, (M, R, hkv, HEAD_DIM))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((M, R, hq), dtype=torch.float32, device=q.device)
    _check(o, "o", torch.bfloat16, q.shape)
    _check(lse, "lse", torch.float32, (M, R, hq))
    nbytes = B.ls_replay_attn_fwd_members_workspace(cache.struct, R, M, hq, num_splits)
    ws = workspace(nbytes, q.device, "fwd")
    B.ls_replay_attn_fwd_members(cache.struct, q.data_ptr(), k_resp.data_ptr(),
                                 v_resp.data_ptr(), R, M, hq, softmax_scale, num_splits,
                                 o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                 _stream(stream))
    return o, lse


def replay_bwd(cache: PagedKVCache, q, k_resp, v_resp, o, lse, d_o, softmax_scale: float,
               num_splits: int, dq=None, dk=None, dv=None, accumulate: bool = False, stream=None):
    R, hq, _ = q.shape
    hkv = cache.num_kv_heads
    for t, n in ((q, "q"), (o, "o"), (d_o, "d_o")):
        _check(t, n, torch.bfloat16, (R, hq, HEAD_DIM))
    _check(k_resp, "k_resp", torch.bfloat16, (R, hkv, HEAD_DIM))
    _check(v_resp, "v_resp", torch.bfloat16, (R, hkv, HEAD_DIM))
    _check(lse, "lse", torch.float32, (R, hq))
    if dq is None:
        dq = torch.empty((R, hq, HEAD_DIM), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty((R, hkv, HEAD_DIM), dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty((R, hkv, HEAD_DIM), dtype=torch.float32, device=q.device)
    _check(dq, "dq", torch.float32, (R, hq, HEAD_DIM))
    _check(dk, "dk", torch.float32, (R, hkv, HEAD_DIM))
    _check(dv, "dv", torch.float32, (R, hkv, HEAD_DIM))
    nbytes = B.ls_replay_attn_bwd_workspace(cache.struct, R, hq, num_splits)
    ws = workspace(nbytes, q.device, "bwd")
    B.ls_replay_attn_bwd(cache.struct, q.data_ptr(), k_resp.data_ptr(), v_resp.data_ptr(),
                         o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), R, hq, softmax_scale,
                         num_splits, int(accumulate), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                         ws.data_ptr(), ws.numel(), _stream(stream))
    return dq, dk, dv


def grpo_loss_fwd_bwd(logits: torch.Tensor, targets: torch.Tensor, logp_old: torch.Tensor,
                      rewards: torch.Tensor, resp_lens: torch.Tensor, member_begin: int,
                      member_end: int, eps: float, adv_eps: float = 1e-6, std_ddof: int = 1,
                      loss: torch.Tensor | None = None, accumulate: bool = False,
                      dlogits: torch.Tensor | None = None, logp_out: torch.Tensor | None = None,
                      stats: torch.Tensor | None = None, stream=None):
    """Returns (loss[1], dlogits, logp[T], stats[4]); loss accumulates when asked."""
    T, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = B.LS_BF16
    elif logits.dtype == torch.float32:
        dt = B.LS_FP32
    else:
        raise ValueError("logits must be bf16 or fp32")
    _check(logits, "logits", logits.dtype)
    _check(targets, "targets", torch.int32, (T,))
    _check(logp_old, "logp_old", torch.float32, (T,))
    G = rewards.numel()
    _check(rewards, "rewards", torch.float32, (G,))
    _check(resp_lens, "resp_lens", torch.int32, (G,))
    dev = logits.device
    if loss is None:
        loss = torch.zeros(1, dtype=torch.float32, device=dev)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    if logp_out is None:
        logp_out = torch.empty(T, dtype=torch.float32, device=dev)
    if stats is None:
        stats = torch.empty(4, dtype=torch.float32, device=dev)
    _check(dlogits, "dlogits", logits.dtype, (T, V))
    nbytes = B.ls_grpo_workspace(T, G)
    ws = workspace(nbytes, dev, "grpo")
    B.ls_grpo_loss_fwd_bwd(logits.data_ptr(), dt, T, V, targets.data_ptr(), logp_old.data_ptr(),
                           rewards.data_ptr(), resp_lens.data_ptr(), G, member_begin, member_end,
                           eps, adv_eps, std_ddof, int(accumulate), loss.data_ptr(),
                           dlogits.data_ptr(), logp_out.data_ptr(), stats.data_ptr(),
                           ws.data_ptr(), ws.numel(), _stream(stream))
    return loss, dlogits, logp_out, stats


def grpo_logp(logits: torch.Tensor, targets: torch.Tensor, ref_logp: torch.Tensor | None = None,
              with_lse: bool = False, stream=None):
    """Pre-step scoring: returns (logp[T], lse[T] or None, kl[T] or None)."""
    T, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = B.LS_BF16
    elif logits.dtype == torch.float32:
        dt = B.LS_FP32
    else:
        raise ValueError("logits must be bf16 or fp32")
    _check(logits, "logits", logits.dtype)
    _check(targets, "targets", torch.int32, (T,))
    dev = logits.device
    logp = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev) if with_lse else None
    kl = None
    if ref_logp is not None:
        _check(ref_logp, "ref_logp", torch.float32, (T,))
        kl = torch.empty(T, dtype=torch.float32, device=dev)
    B.ls_grpo_logp(logits.data_ptr(), dt, T, V, targets.data_ptr(),
                   ref_logp.data_ptr() if ref_logp is not None else None, logp.data_ptr(),
                   lse.data_ptr() if lse is not None else None,
                   kl.data_ptr() if kl is not None else None, _stream(stream))
    return logp, lse, kl


def replay_fwd_ragged(cache: PagedKVCache, q: torch.Tensor, k_resp: torch.Tensor,
                      v_resp: torch.Tensor, lens, softmax_scale: float, num_splits: int,
                      o: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Forward of ragged members laid out back to back: q [T][Hq][128], k_resp / v_resp
    [T][Hkv][128], lens the members' lengths (summing to T)."""
    T, hq, _ = q.shape
    lens = [int(x) for x in lens]
    if sum(lens) != T:
        raise ValueError("member lengths must add up to the token count")
    _check(q, "q", torch.bfloat16, (T, hq, HEAD_DIM))
    _check(k_resp, "k_resp", torch.bfloat16, (T, cache.num_kv_heads, HEAD_DIM))
    _check(v_resp, "v_resp", torch.bfloat16, (T, cache.num_kv_heads, HEAD_DIM))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    nbytes = B.ls_replay_attn_fwd_ragged_workspace(cache.struct, lens, hq, num_splits)
    ws = workspace(nbytes, q.device, "fwd")
    B.ls_replay_attn_fwd_ragged(cache.struct, q.data_ptr(), k_resp.data_ptr(), v_resp.data_ptr(),
                                lens, hq, softmax_scale, num_splits, o.data_ptr(), lse.data_ptr(),
                                ws.data_ptr(), ws.numel(), _stream(stream))
    return o, lse


def replay_bwd_ragged(cache: PagedKVCache, q, k_resp, v_resp, o, lse, d_o, lens,
                      softmax_scale: float, num_splits: int, dq=None, dk=None, dv=None,
                      accumulate: bool = False, stream=None):
    """Backward of ragged members laid out back to back (see replay_fwd_ragged)."""
    T, hq, _ = q.shape
    hkv = cache.num_kv_heads
    lens = [int(x) for x in lens]
    if sum(lens) != T:
        raise ValueError("member lengths must add up to the token count")
    for t, n in ((q, "q"), (o, "o"), (d_o, "d_o")):
        _check(t, n, torch.bfloat16, (T, hq, HEAD_DIM))
    _check(lse, "lse", torch.float32, (T, hq))
    dev = q.device
    if dq is None:
        dq = torch.empty((T, hq, HEAD_DIM), dtype=torch.float32, device=dev)
    if dk is None:
        dk = torch.empty((T, hkv, HEAD_DIM), dtype=torch.float32, device=dev)
    if dv is None:
        dv = torch.empty((T, hkv, HEAD_DIM), dtype=torch.float32, device=dev)
    nbytes = B.ls_replay_attn_bwd_ragged_workspace(cache.struct, lens, hq, num_splits)
    ws = workspace(nbytes, dev, "bwd")
    B.ls_replay_attn_bwd_ragged(cache.struct, q.data_ptr(), k_resp.data_ptr(), v_resp.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), lens, hq,
                                softmax_scale, num_splits, int(accumulate), dq.data_ptr(),
                                dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), ws.numel(),
                                _stream(stream))
    return dq, dk, dv


def gdn_replay_fwd(state0: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   g: torch.Tensor, beta: torch.Tensor, scale: float, o: torch.Tensor | None = None,
                   state_out: torch.Tensor | None = None, with_state: bool = False, stream=None):
    """Gated-DeltaNet replay of R tokens from a captured state: state0 fp32 [H][128][128],
    q/k/v bf16 [R][H][128], g/beta fp32 [R][H].  Returns (o, state_out or None)."""
    R, H, _ = q.shape
    _check(state0, "state0", torch.float32, (H, HEAD_DIM, HEAD_DIM))
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, (R, H, HEAD_DIM))
    _check(g, "g", torch.float32, (R, H))
    _check(beta, "beta", torch.float32, (R, H))
    if o is None:
        o = torch.empty_like(q)
    if state_out is None and with_state:
        state_out = torch.empty_like(state0)
    nbytes = B.ls_gdn_replay_fwd_workspace(R, H)
    ws = workspace(nbytes, q.device, "gdn")
    B.ls_gdn_replay_fwd(state0.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                        beta.data_ptr(), R, H, scale, o.data_ptr(),
                        state_out.data_ptr() if state_out is not None else None, ws.data_ptr(),
                        ws.numel(), _stream(stream))
    return o, state_out


def gdn_replay_bwd(state0, q, k, v, g, beta, d_o, scale: float, grads=None,
                   accumulate: bool = False, stream=None):
    """Gradients (dq, dk, dv, dg, dbeta) of the replay with the captured state stopgrad."""
    R, H, _ = q.shape
    _check(d_o, "d_o", torch.bfloat16, (R, H, HEAD_DIM))
    if grads is None:
        dev = q.device
        grads = (torch.empty((R, H, HEAD_DIM), dtype=torch.float32, device=dev),
                 torch.empty((R, H, HEAD_DIM), dtype=torch.float32, device=dev),
                 torch.empty((R, H, HEAD_DIM), dtype=torch.float32, device=dev),
                 torch.empty((R, H), dtype=torch.float32, device=dev),
                 torch.empty((R, H), dtype=torch.float32, device=dev))
    dq, dk, dv, dg, db = grads
    nbytes = B.ls_gdn_replay_bwd_workspace(R, H)
    ws = workspace(nbytes, q.device, "gdn")
    B.ls_gdn_replay_bwd(state0.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                        beta.data_ptr(), d_o.data_ptr(), R, H, scale, int(accumulate),
                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), db.data_ptr(),
                        ws.data_ptr(), ws.numel(), _stream(stream))
    return dq, dk, dv, dg, db


def last_device_error(stream=None) -> int:
    return B.ls_last_device_error(_stream(stream))


# ---------------------------------------------------------------- latent (MLA) replay

LATENT_DIM = 512           # c_j: the values attention averages
LATENT_ROW = 576           # c_j followed by the 64-value rotary key


class LatentCache:
    """Latent (MLA-style) pages of one layer plus page table (ls_latent_cache): rows of
    LATENT_ROW bf16 values shared by all heads.  host_pool=True places the pool in pinned
    host memory (Grace memory on a Grace-Blackwell node), read there by the kernels."""

    def __init__(self, num_pages: int, page_table: torch.Tensor, page_size: int, num_tokens: int,
                 device=None, fill: float | None = None, pool: torch.Tensor | None = None,
                 host_pool: bool = False):
        device = torch.device(device) if device is not None else page_table.device
        shape = (num_pages, page_size, LATENT_ROW)
        if pool is None:
            pool = (torch.empty(shape, dtype=torch.bfloat16, pin_memory=True) if host_pool
                    else torch.empty(shape, dtype=torch.bfloat16, device=device))
            if fill is not None:
                pool.fill_(fill)
        _check_pool(pool, "pool", shape)
        _check(page_table, "page_table", torch.int32)
        self.pool, self.page_table = pool, page_table
        self.page_size, self.num_tokens = page_size, num_tokens
        self.struct = B.ls_latent_cache(pool.data_ptr(), page_table.data_ptr(), num_pages,
                                        page_table.numel(), page_size, num_tokens)

    @property
    def device(self):
        return self.page_table.device

    def capture(self, lat: torch.Tensor, start_pos: int = 0, stream=None) -> None:
        n = lat.shape[0]
        _check(lat, "lat", torch.bfloat16, (n, LATENT_ROW))
        B.ls_capture_latent(self.struct, lat.data_ptr(), start_pos, n, _stream(stream))


def mla_replay_fwd(cache: LatentCache, q: torch.Tensor, lat_resp: torch.Tensor,
                   softmax_scale: float, num_splits: int, o: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, stream=None):
    """q [R][H][576] absorbed queries, lat_resp [R][576] the response's own rows ->
    o [R][H][512] (bf16), lse [R][H] (fp32)."""
    R, H, _ = q.shape
    _check(q, "q", torch.bfloat16, (R, H, LATENT_ROW))
    _check(lat_resp, "lat_resp", torch.bfloat16, (R, LATENT_ROW))
    if o is None:
        o = torch.empty((R, H, LATENT_DIM), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((R, H), dtype=torch.float32, device=q.device)
    _check(o, "o", torch.bfloat16, (R, H, LATENT_DIM))
    _check(lse, "lse", torch.float32, (R, H))
    nbytes = B.ls_mla_replay_fwd_workspace(cache.struct, R, H, num_splits)
    ws = workspace(nbytes, q.device, "mla_fwd")
    B.ls_mla_replay_fwd(cache.struct, q.data_ptr(), lat_resp.data_ptr(), R, H, softmax_scale,
                        num_splits, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                        _stream(stream))
    return o, lse


def mla_replay_bwd(cache: LatentCache, q: torch.Tensor, lat_resp: torch.Tensor, o: torch.Tensor,
                   lse: torch.Tensor, d_o: torch.Tensor, softmax_scale: float, num_splits: int,
                   dq: torch.Tensor | None = None, dlat: torch.Tensor | None = None, stream=None):
    """Backward of mla_replay_fwd with the prompt rows stopgrad: o, lse from the forward,
    d_o [R][H][512] bf16 -> dq [R][H][576] and dlat [R][576] (fp32, the gradient of the
    response's own rows)."""
    R, H, _ = q.shape
    _check(q, "q", torch.bfloat16, (R, H, LATENT_ROW))
    _check(lat_resp, "lat_resp", torch.bfloat16, (R, LATENT_ROW))
    _check(o, "o", torch.bfloat16, (R, H, LATENT_DIM))
    _check(lse, "lse", torch.float32, (R, H))
    _check(d_o, "d_o", torch.bfloat16, (R, H, LATENT_DIM))
    if dq is None:
        dq = torch.empty((R, H, LATENT_ROW), dtype=torch.float32, device=q.device)
    if dlat is None:
        dlat = torch.empty((R, LATENT_ROW), dtype=torch.float32, device=q.device)
    _check(dq, "dq", torch.float32, (R, H, LATENT_ROW))
    _check(dlat, "dlat", torch.float32, (R, LATENT_ROW))
    nbytes = B.ls_mla_replay_bwd_workspace(cache.struct, R, H, num_splits)
    ws = workspace(nbytes, q.device, "mla_bwd")
    B.ls_mla_replay_bwd(cache.struct, q.data_ptr(), lat_resp.data_ptr(), o.data_ptr(),
                        lse.data_ptr(), d_o.data_ptr(), R, H, softmax_scale, num_splits,
                        dq.data_ptr(), dlat.data_ptr(), ws.data_ptr(), ws.numel(),
                        _stream(stream))
    return dq, dlat


# ---------------------------------------------------------------- query / key stage
#
# These calls are a few microseconds of GPU work at decode sizes, so their argument checks
# are kept to one pass over each tensor's attributes.  With a stream given, a call does
# what it does with that stream as the current one: what it allocates belongs to it.

def _as_current(stream):
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(h) if h > 1 else torch.cuda.default_stream())


def _dev_stream(dev: int) -> int:
    """The current stream of CUDA device `dev`, which has to be the current one (the
    kernels run there)."""
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if dev != torch.cuda.current_device():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _refuse(t: torch.Tensor, name: str, dtype, shape, dev: int):
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, others on cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of the given type, shape and device."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype, shape, dev: int):
    """(address, token stride, head stride) of a [T][H][128] tensor whose heads are dense
    rows; token and head strides are free, in whole 16-byte units."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, dtype, shape, dev)
    ts, hs, es = t.stride()
    if (es != 1 or (ts | hs) & 7) and t.numel():
        raise ValueError(f"{name}: heads must be contiguous, at strides of whole 8 elements")
    return t.data_ptr(), ts, hs


def _no_overlap(t: torch.Tensor, name: str):
    """Rows of an output, written at the same time, must be distinct memory."""
    T, H, _ = t.shape
    st, sh = t.stride(0), t.stride(1)
    if H > 1 and sh < HEAD_DIM or T > 1 and st < HEAD_DIM:
        raise ValueError(f"{name}: rows overlap")
    if T > 1 and H > 1 and st < (H - 1) * sh + HEAD_DIM and sh < (T - 1) * st + HEAD_DIM:
        raise ValueError(f"{name}: rows overlap")


def _out_rows(t, like: torch.Tensor, name: str, shape, dev: int):
    """An output of the stage: allocated dense, or the caller's rows."""
    if t is None:
        t = torch.empty(shape, dtype=torch.bfloat16, device=like.device)
        return t, (t.data_ptr(), shape[1] * HEAD_DIM, HEAD_DIM)
    r = _rows(t, name, torch.bfloat16, shape, dev)
    _no_overlap(t, name)
    return t, r


_NO_ROWS = (None, 0, 0)


def _view(q, k=_NO_ROWS, v=_NO_ROWS) -> B.ls_qkv_view:
    return B.ls_qkv_view(q[0], k[0], v[0], q[1], q[2], k[1], k[2], v[1], v[2])


class Rotary:
    """Rotary positions of a layer (ls_rotary): inv_freq fp64 [rot_dim / 2], radians per
    position; with more than one axis, pair_axis int32 [rot_dim / 2] gives each pair's.
    Pairs are (j, j + rot_dim / 2), or (2 j, 2 j + 1) when interleaved."""

    def __init__(self, inv_freq: torch.Tensor, pair_axis: torch.Tensor | None = None, axes: int = 1,
                 interleaved: bool = False):
        _check(inv_freq, "inv_freq", torch.float64)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must have one dimension")
        if pair_axis is not None:
            _check(pair_axis, "pair_axis", torch.int32, inv_freq.shape)
            if pair_axis.device != inv_freq.device:
                raise ValueError("pair_axis and inv_freq must be on one device")
        elif axes > 1:
            raise ValueError("pair_axis is required with more than one axis")
        self.inv_freq, self.pair_axis, self.axes = inv_freq, pair_axis, axes
        self.rot_dim, self.interleaved = 2 * inv_freq.numel(), interleaved
        self.device_index = inv_freq.get_device()
        self.struct = B.ls_rotary(inv_freq.data_ptr(),
                                  pair_axis.data_ptr() if pair_axis is not None else None,
                                  self.rot_dim, axes, int(interleaved))

    @classmethod
    def from_base(cls, base: float, rot_dim: int, device, **kw) -> "Rotary":
        """inv_freq[j] = base^(-2 j / rot_dim)."""
        j = torch.arange(rot_dim // 2, dtype=torch.float64)
        return cls((float(base) ** (-2.0 * j / rot_dim)).to(device), **kw)


def _stage_args(q, k, positions, rotary, wq, wk, norm, eps, weight_offset):
    """Checks shared by the calls of the stage; returns (device, T, Hq, Hkv, q rows, k rows,
    norm struct, rotary struct, positions address)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T][H][128]")
    dev = q.get_device()
    T, hq, _ = q.shape
    hkv = k.shape[1]
    qr = _rows(q, "q", torch.bfloat16, (T, hq, HEAD_DIM), dev)
    kr = _rows(k, "k", torch.bfloat16, (T, hkv, HEAD_DIM), dev)
    ns = None
    if norm:
        dt = torch.float32 if wq is None and wk is None else (wk if wq is None else wq).dtype
        if dt is not torch.float32 and dt is not torch.bfloat16:
            raise ValueError("wq and wk must both be fp32 or both bf16")
        ns = B.ls_qk_norm(_dense(wq, "wq", dt, (HEAD_DIM,), dev) if wq is not None else None,
                          _dense(wk, "wk", dt, (HEAD_DIM,), dev) if wk is not None else None,
                          B.LS_FP32 if dt is torch.float32 else B.LS_BF16, weight_offset, eps)
    elif wq is not None or wk is not None:
        raise ValueError("norm weights without a norm")
    if rotary is None:
        return dev, T, hq, hkv, qr, kr, ns, None, None
    if positions is None:
        raise ValueError("positions are required with rotary")
    if rotary.device_index != dev:
        raise ValueError("the rotary frequencies are on another device")
    shape = (T,) if rotary.axes == 1 and positions.dim() == 1 else (rotary.axes, T)
    return (dev, T, hq, hkv, qr, kr, ns, rotary.struct,
            _dense(positions, "positions", torch.int32, shape, dev))


def qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor | None,
                     positions: torch.Tensor | None, rotary: Rotary | None,
                     wq: torch.Tensor | None = None, wk: torch.Tensor | None = None,
                     norm: bool = True, eps: float = 1e-6, weight_offset: float = 0.0,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     v_out: torch.Tensor | None = None, stream=None):
    """Norm of every query and key head and rotary positions in one pass: q [T][Hq][128],
    k / v [T][Hkv][128] bf16, any token and head strides (slices of a packed projection),
    positions int32 [axes][T].  Returns (q_out, k_out, v_out); the outputs are dense
    unless given (an output may be its input), v is copied into the replay's layout."""
    if stream is not None:
        with _as_current(stream):
            return qk_norm_rope_fwd(q, k, v, positions, rotary, wq, wk, norm, eps, weight_offset,
                                    q_out, k_out, v_out)
    dev, T, hq, hkv, qr, kr, ns, rs, pp = _stage_args(q, k, positions, rotary, wq, wk, norm, eps,
                                                      weight_offset)
    st = _dev_stream(dev)
    qs, ks = (T, hq, HEAD_DIM), (T, hkv, HEAD_DIM)
    vr = vo = _NO_ROWS
    if v is not None:
        vr = _rows(v, "v", torch.bfloat16, ks, dev)
        v_out, vo = _out_rows(v_out, q, "v_out", ks, dev)
    elif v_out is not None:
        raise ValueError("v_out without v")
    q_out, qo = _out_rows(q_out, q, "q_out", qs, dev)
    k_out, ko = _out_rows(k_out, q, "k_out", ks, dev)
    B.ls_qk_norm_rope_fwd(_view(qr, kr, vr), T, hq, hkv, ns, rs, pp, _view(qo, ko, vo), st)
    return q_out, k_out, v_out


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor | None,
                     rotary: Rotary | None, dq: torch.Tensor, dk: torch.Tensor,
                     dv: torch.Tensor | None = None, wq: torch.Tensor | None = None,
                     wk: torch.Tensor | None = None, norm: bool = True, eps: float = 1e-6,
                     weight_offset: float = 0.0, dx_q: torch.Tensor | None = None,
                     dx_k: torch.Tensor | None = None, dx_v: torch.Tensor | None = None,
                     dwq: torch.Tensor | None = None, dwk: torch.Tensor | None = None,
                     accumulate: bool = False, stream=None):
    """Backward of qk_norm_rope_fwd: q, k its inputs; dq, dk, dv the gradients of its
    outputs (all fp32, as the replay backward gives them, or all bf16).  Returns (dx_q,
    dx_k, dx_v, dwq, dwk): bf16 gradients of the inputs (dense unless given, e.g. as
    slices of the packed projection's gradient) and fp32 [128] weight gradients, which
    accumulate adds into; a weight gradient is returned for each weight given."""
    if stream is not None:
        with _as_current(stream):
            return qk_norm_rope_bwd(q, k, positions, rotary, dq, dk, dv, wq, wk, norm, eps,
                                    weight_offset, dx_q, dx_k, dx_v, dwq, dwk, accumulate)
    dev, T, hq, hkv, qr, kr, ns, rs, pp = _stage_args(q, k, positions, rotary, wq, wk, norm, eps,
                                                      weight_offset)
    st = _dev_stream(dev)
    dt = dq.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise ValueError("dq must be fp32 or bf16")
    qs, ks = (T, hq, HEAD_DIM), (T, hkv, HEAD_DIM)
    gq, gk, gv, ov = _rows(dq, "dq", dt, qs, dev), _rows(dk, "dk", dt, ks, dev), _NO_ROWS, _NO_ROWS
    if dv is not None:
        gv = _rows(dv, "dv", dt, ks, dev)
        dx_v, ov = _out_rows(dx_v, q, "dx_v", ks, dev)
    elif dx_v is not None:
        raise ValueError("dx_v without dv")
    dx_q, oq = _out_rows(dx_q, q, "dx_q", qs, dev)
    dx_k, ok = _out_rows(dx_k, q, "dx_k", ks, dev)
    if not norm and (dwq is not None or dwk is not None):
        raise ValueError("weight gradients without a norm")
    if accumulate and ((wq is not None and dwq is None) or (wk is not None and dwk is None)):
        raise ValueError("accumulate needs the weight gradients to add into")
    if wq is not None and dwq is None:
        dwq = torch.empty(HEAD_DIM, dtype=torch.float32, device=q.device)
    if wk is not None and dwk is None:
        dwk = torch.empty(HEAD_DIM, dtype=torch.float32, device=q.device)
    pq = pk = None
    if dwq is not None:
        pq = _dense(dwq, "dwq", torch.float32, (HEAD_DIM,), dev)
    if dwk is not None:
        pk = _dense(dwk, "dwk", torch.float32, (HEAD_DIM,), dev)
    _with_workspace(B.ls_qk_norm_rope_bwd,
                    (_view(qr, kr), T, hq, hkv, ns, rs, pp, _view(gq, gk, gv),
                     B.LS_FP32 if dt is torch.float32 else B.LS_BF16, int(accumulate),
                     _view(oq, ok, ov), pq, pk),
                    lambda: B.ls_qk_norm_rope_bwd_workspace(T), q, "qk_norm", st)
    return dx_q, dx_k, dx_v, dwq, dwk


class PagePool:
    """K / V pages of one layer (ls_page_pool): bf16 [num_pages][Hkv][page_size][128]."""

    def __init__(self, k_pool: torch.Tensor, v_pool: torch.Tensor):
        if k_pool.dim() != 4:
            raise ValueError("k_pool must be [num_pages][Hkv][page_size][128]")
        n, hkv, ps, _ = k_pool.shape
        _check_pool(k_pool, "k_pool", (n, hkv, ps, HEAD_DIM))
        _check_pool(v_pool, "v_pool", (n, hkv, ps, HEAD_DIM))
        self.k_pool, self.v_pool = k_pool, v_pool
        self.num_pages, self.num_kv_heads, self.page_size = n, hkv, ps
        # -1: pinned host memory, read and written there from any device
        self.device_indices = {k_pool.get_device(), v_pool.get_device()} - {-1}
        self.struct = B.ls_page_pool(k_pool.data_ptr(), v_pool.data_ptr(), n, ps, hkv, HEAD_DIM)

    @classmethod
    def empty(cls, num_pages: int, num_kv_heads: int, page_size: int, device) -> "PagePool":
        shape = (num_pages, num_kv_heads, page_size, HEAD_DIM)
        return cls(torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.empty(shape, dtype=torch.bfloat16, device=device))

    @classmethod
    def of(cls, cache: PagedKVCache) -> "PagePool":
        """The pools of a prompt cache, to append a chunk of the prompt to by slot."""
        return cls(cache.k_pool, cache.v_pool)


def qk_norm_rope_append(pool: PagePool, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        slots: torch.Tensor, positions: torch.Tensor | None, rotary: Rotary | None,
                        wq: torch.Tensor | None = None, wk: torch.Tensor | None = None,
                        norm: bool = True, eps: float = 1e-6, weight_offset: float = 0.0,
                        q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qk_norm_rope_fwd with keys and values written into `pool` at slots[t] = page *
    page_size + offset (int32 [T]; negative: a padding token, nothing of it is written).
    Returns q_out."""
    if stream is not None:
        with _as_current(stream):
            return qk_norm_rope_append(pool, q, k, v, slots, positions, rotary, wq, wk, norm, eps,
                                       weight_offset, q_out)
    dev, T, hq, hkv, qr, kr, ns, rs, pp = _stage_args(q, k, positions, rotary, wq, wk, norm, eps,
                                                      weight_offset)
    st = _dev_stream(dev)
    if hkv != pool.num_kv_heads or pool.device_indices - {dev}:
        raise ValueError("the pool has other key heads or is on another device")
    vr = _rows(v, "v", torch.bfloat16, (T, hkv, HEAD_DIM), dev)
    sp = _dense(slots, "slots", torch.int32, (T,), dev)
    q_out, qo = _out_rows(q_out, q, "q_out", (T, hq, HEAD_DIM), dev)
    B.ls_qk_norm_rope_append(pool.struct, _view(qr, kr, vr), T, hq, ns, rs, pp, sp, _view(qo), st)
    return q_out


# ---------------------------------------------------------------- decode step

class PageAllocator:
    """Pages of a group's growing responses (ls_extend_pages): block_table int32
    [members][max_blocks], lens int32 [members] (negative: out of use), free_list int32
    [num_free] and used int32 [1], all on the GPU; for branching responses also shared int32
    [num_pages], the owners of each page besides the first (zeros at the start).  One
    allocator serves every layer's pools: the token -> page map is the same in each."""

    def __init__(self, block_table: torch.Tensor, lens: torch.Tensor, free_list: torch.Tensor,
                 used: torch.Tensor, page_size: int, num_pages: int | None = None,
                 shared: torch.Tensor | None = None):
        _check(block_table, "block_table", torch.int32)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [members][max_blocks]")
        _check(lens, "lens", torch.int32, block_table.shape[:1])
        _check(free_list, "free_list", torch.int32, (free_list.numel(),))
        _check(used, "used", torch.int32, (1,))
        for t in (lens, free_list, used):
            if t.device != block_table.device:
                raise ValueError("the allocator's tensors must be on one device")
        self.block_table, self.lens, self.free_list, self.used = block_table, lens, free_list, used
        self.page_size = page_size
        self.members, self.max_blocks = block_table.shape
        self.num_free = free_list.numel()
        self.num_pages = self.num_free if num_pages is None else num_pages
        if shared is not None:
            _check(shared, "shared", torch.int32, (self.num_pages,))
            if shared.device != block_table.device:
                raise ValueError("the allocator's tensors must be on one device")
        self.shared = shared
        self.device_index = block_table.get_device()

    @classmethod
    def empty(cls, members: int, max_blocks: int, num_pages: int, page_size: int,
              device, sharing: bool = False) -> "PageAllocator":
        """No tokens yet, every page of the pool free; sharing: pages may have several owners
        (fork_pages)."""
        z = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((members, max_blocks), **z), torch.zeros(members, **z),
                   torch.arange(num_pages, **z), torch.zeros(1, **z), page_size,
                   shared=torch.zeros(num_pages, **z) if sharing else None)


def extend_pages(alloc: PageAllocator, add: torch.Tensor | None, pos0: int, slots: torch.Tensor,
                 positions: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
                 used_out: torch.Tensor | None = None, stream=None,
                 member_rows: int | None = None, added: torch.Tensor | None = None) -> None:
    """Room for add[m] more tokens of every member: fills slots int32 [capacity] (-1 behind
    the last token) and positions int32 [axes][capacity] (pos0 + index within the
    response), enters new pages into the table and advances alloc.lens and alloc.used (or
    writes them to lens_out / used_out).  See ls_extend_pages for what is refused.

    The tokens are packed, member after member; with member_rows given, capacity is members *
    member_rows and a member's tokens are the last of its own rows (-1 before them), the order
    in which decode_attn takes queries [members][member_rows] while some members add none.

    With added int32 [members] (and member_rows; see ls_extend_drafts) it says what each member got,
    0 of a refused call; add None then means all rows of every member in use."""
    if stream is not None:
        with _as_current(stream):
            return extend_pages(alloc, add, pos0, slots, positions, lens_out, used_out,
                                member_rows=member_rows, added=added)
    if not -2 ** 31 <= pos0 < 2 ** 31:  # a C int would take its low bits
        raise ValueError(f"pos0 must be a position, got {pos0}")
    M, dev, i32 = alloc.members, alloc.device_index, torch.int32
    st = _dev_stream(dev)
    cap = slots.shape[0] if slots.dim() == 1 else -1
    if member_rows is not None and (member_rows < 1 or cap != M * member_rows):
        raise ValueError(f"slots must be [{M} members * member_rows], member_rows at least 1")
    if added is None and add is None or added is not None and member_rows is None:
        raise ValueError("counts that are left out need added, and added member_rows")
    sp = _dense(slots, "slots", i32, (cap,), dev)
    axes, pp = 1, None
    if positions is not None:
        axes = positions.shape[0] if positions.dim() == 2 else -1
        pp = _dense(positions, "positions", i32, (axes, cap), dev)
    lens, used = alloc.lens.data_ptr(), alloc.used.data_ptr()
    call, room = ((B.ls_extend_pages, cap) if member_rows is None
                  else (B.ls_extend_pages_by_member, member_rows) if added is None
                  else (B.ls_extend_drafts, member_rows))
    more = () if added is None else (_dense(added, "added", i32, (M,), dev),)
    call(alloc.block_table.data_ptr(), M, alloc.max_blocks, alloc.page_size,
         alloc.num_pages, lens, None if add is None else _dense(add, "add", i32, (M,), dev),
         alloc.free_list.data_ptr(), alloc.num_free, used, pos0, axes, room, sp, pp,
         lens if lens_out is None else _dense(lens_out, "lens_out", i32, (M,), dev),
         used if used_out is None else _dense(used_out, "used_out", i32, (1,), dev), *more, st)


class ResponseCache:
    """One layer's view of a group's responses (ls_resp_cache): its page pool under the
    members' block table and lengths (an allocator's, shared by all layers)."""

    def __init__(self, pool: PagePool, block_table: torch.Tensor, lens: torch.Tensor):
        _check(block_table, "block_table", torch.int32)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [members][max_blocks]")
        _check(lens, "lens", torch.int32, block_table.shape[:1])
        if lens.device != block_table.device:
            raise ValueError("block_table and lens must be on one device")
        self.pool, self.block_table, self.lens = pool, block_table, lens
        self.members = block_table.shape[0]
        self.device_index = block_table.get_device()
        if pool.device_indices - {self.device_index}:
            raise ValueError("the pool is on another device")
        self.struct = B.ls_resp_cache(pool.struct, block_table.data_ptr(), lens.data_ptr(),
                                      block_table.shape[0], block_table.shape[1])

    @classmethod
    def of(cls, pool: PagePool, alloc: PageAllocator) -> "ResponseCache":
        if pool.page_size != alloc.page_size or pool.num_pages < alloc.num_pages:
            raise ValueError("the pool does not hold the allocator's pages")
        return cls(pool, alloc.block_table, alloc.lens)


def _decode_args(cache: PagedKVCache, resp: ResponseCache, q: torch.Tensor, o, lse):
    """Checks shared by the decode calls; returns (members, n, Hq, device, stream, q's address, o,
    lse, their addresses)."""
    if q.dim() != 4:
        raise ValueError("q must be [members][n][Hq][128]")
    _, n, hq, _ = shape = q.shape
    M, dev = resp.members, resp.device_index
    st = _dev_stream(dev)
    if (cache.page_table.get_device() != dev or cache.k_pool.get_device() not in (-1, dev)
            or cache.v_pool.get_device() not in (-1, dev)):
        raise ValueError("the prompt's pages are on another device")
    qp = _dense(q, "q", torch.bfloat16, (M, n, hq, HEAD_DIM), dev)
    if o is None:
        o = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((M, n, hq), dtype=torch.float32, device=q.device)
    op = _dense(o, "o", torch.bfloat16, shape, dev)
    lp = _dense(lse, "lse", torch.float32, (M, n, hq), dev)
    return M, n, hq, dev, st, qp, o, lse, op, lp


def decode_attn(cache: PagedKVCache, resp: ResponseCache, q: torch.Tensor, softmax_scale: float,
                o: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention of a decode step: q [members][n][Hq][128], the n newest tokens of every
    member (already appended to its pages), over the shared prompt and the member's own
    response.  Returns (o, lse)."""
    if stream is not None:
        with _as_current(stream):
            return decode_attn(cache, resp, q, softmax_scale, o, lse)
    M, n, hq, dev, st, qp, o, lse, op, lp = _decode_args(cache, resp, q, o, lse)
    _with_workspace(B.ls_decode_attn, (cache.struct, resp.struct, qp, n, hq, softmax_scale, op, lp),
                    lambda: B.ls_decode_attn_workspace(cache.struct, resp.struct, n, hq), q,
                    "decode", st)
    return o, lse


# ---------------------------------------------------------------- drafted trees

def _draft_args(parents, lens, drafted):
    """(members, n, device, parents' address, lens', drafted's) of a step's draft."""
    if parents.dim() != 2:
        raise ValueError("parents must be [members][n]")
    M, n = parents.shape
    dev = parents.get_device()
    return (M, n, dev, _dense(parents, "parents", torch.int32, (M, n), dev),
            _dense(lens, "lens", torch.int32, (M,), dev),
            None if drafted is None else _dense(drafted, "drafted", torch.int32, (M,), dev))


def draft_tree(parents: torch.Tensor, lens: torch.Tensor, pos0: int,
               drafted: torch.Tensor | None = None, axes: int = 1,
               visible: torch.Tensor | None = None, positions: torch.Tensor | None = None,
               stream=None):
    """The plan of a step over drafted trees (ls_draft_tree): parents int32 [members][n] (the row
    that a row's node continues, -1: the context), lens int32 [members] with the drafts in them,
    drafted int32 [members] (default: n of each; the last rows).  Returns (visible int32
    [members][n][ceil(n / 32)], the rows that a row sees, and positions int32
    [axes][members][n], pos0 + context + depth)."""
    if stream is not None:
        with _as_current(stream):
            return draft_tree(parents, lens, pos0, drafted, axes, visible, positions)
    M, n, dev, pp, lp, dp = _draft_args(parents, lens, drafted)
    st = _dev_stream(dev)
    if not 0 <= pos0 < 2 ** 31:
        raise ValueError(f"pos0 must be a position, got {pos0}")
    if visible is None:
        visible = torch.empty((M, n, (n + 31) // 32), dtype=torch.int32, device=parents.device)
    if positions is None:
        positions = torch.empty((axes, M, n), dtype=torch.int32, device=parents.device)
    elif positions.dim() == 3:
        axes = positions.shape[0]
    B.ls_draft_tree(pp, lp, dp, M, n, pos0, axes,
                    _dense(visible, "visible", torch.int32, (M, n, (n + 31) // 32), dev),
                    _dense(positions, "positions", torch.int32, (axes, M, n), dev), st)
    return visible, positions


def decode_attn_tree(cache: PagedKVCache, resp: ResponseCache, q: torch.Tensor,
                     visible: torch.Tensor, softmax_scale: float,
                     drafted: torch.Tensor | None = None, o: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, stream=None):
    """decode_attn of drafted trees: q [members][n][Hq][128], row r of member m over the prompt,
    the member's context and the drafted rows of visible[m][r] (draft_tree's).  Rows before the
    last drafted[m] are padding and stay as they are in o and lse.  Returns (o, lse)."""
    if stream is not None:
        with _as_current(stream):
            return decode_attn_tree(cache, resp, q, visible, softmax_scale, drafted, o, lse)
    M, n, hq, dev, st, qp, o, lse, op, lp = _decode_args(cache, resp, q, o, lse)
    vp = _dense(visible, "visible", torch.int32, (M, n, (n + 31) // 32), dev)
    dp = None if drafted is None else _dense(drafted, "drafted", torch.int32, (M,), dev)
    _with_workspace(B.ls_decode_attn_tree,
                    (cache.struct, resp.struct, qp, n, hq, vp, dp, softmax_scale, op, lp),
                    lambda: B.ls_decode_attn_tree_workspace(cache.struct, resp.struct, n, hq), q,
                    "decode", st)
    return o, lse


def accept_draft(parents: torch.Tensor, tokens: torch.Tensor, chosen: torch.Tensor,
                 lens: torch.Tensor, drafted: torch.Tensor | None = None, stream=None):
    """The path of each member's draft that the policy chooses itself (ls_accept_draft): tokens
    int32 [members][n] drafted, chosen int32 [members][n] the policy's token behind each row.
    Returns (rows int32 [members][n], the kept rows, -1 behind them; count [members]; follow
    [members], the token chosen behind the last kept row; ends [members], the members' lengths
    with the kept rows)."""
    if stream is not None:
        with _as_current(stream):
            return accept_draft(parents, tokens, chosen, lens, drafted)
    M, n, dev, pp, lp, dp = _draft_args(parents, lens, drafted)
    st = _dev_stream(dev)
    tp = _dense(tokens, "tokens", torch.int32, (M, n), dev)
    cp = _dense(chosen, "chosen", torch.int32, (M, n), dev)
    rows = torch.empty((M, n), dtype=torch.int32, device=parents.device)
    count, follow, ends = (torch.empty_like(lens) for _ in range(3))
    B.ls_accept_draft(pp, tp, cp, lp, dp, M, n, rows.data_ptr(), count.data_ptr(),
                      follow.data_ptr(), ends.data_ptr(), st)
    return rows, count, follow, ends


class LayerPools:
    """The K / V pages of every layer under one block table: bf16
    [layers][num_pages][Hkv][page_size][128] each, for calls that move rows in all of them."""

    def __init__(self, k_pools: torch.Tensor, v_pools: torch.Tensor):
        if k_pools.dim() != 5 or k_pools.shape[0] < 1:
            raise ValueError("k_pools must be [layers][num_pages][Hkv][page_size][128]")
        L, n, hkv, ps, _ = k_pools.shape
        _check_pool(k_pools, "k_pools", (L, n, hkv, ps, HEAD_DIM))
        _check_pool(v_pools, "v_pools", (L, n, hkv, ps, HEAD_DIM))
        self.k_pools, self.v_pools = k_pools, v_pools
        self.layers, self.num_pages, self.page_size = L, n, ps
        self.layer_stride = n * hkv * ps * HEAD_DIM
        self.device_indices = {k_pools.get_device(), v_pools.get_device()} - {-1}
        self.struct = B.ls_page_pool(k_pools.data_ptr(), v_pools.data_ptr(), n, ps, hkv, HEAD_DIM)


def _of_alloc(pools: LayerPools, alloc: PageAllocator):
    if (pools.page_size != alloc.page_size or pools.num_pages < alloc.num_pages
            or pools.device_indices - {alloc.device_index}):
        raise ValueError("the pools do not hold the allocator's pages")


def compact_rows(alloc: PageAllocator, pools: LayerPools, rows: torch.Tensor, count: torch.Tensor,
                 drafted: torch.Tensor | None = None, stream=None) -> None:
    """The keys and values of accept_draft's rows follow the members' contexts, one behind the
    other, in every layer's pages.  alloc.lens still counts the drafts; trim_pages to
    accept_draft's ends comes next."""
    if stream is not None:
        with _as_current(stream):
            return compact_rows(alloc, pools, rows, count, drafted)
    M, dev = alloc.members, alloc.device_index
    st = _dev_stream(dev)
    _of_alloc(pools, alloc)
    n = rows.shape[1] if rows.dim() == 2 else -1
    B.ls_compact_rows(pools.struct, pools.layers, pools.layer_stride, alloc.block_table.data_ptr(),
                      alloc.max_blocks, alloc.lens.data_ptr(),
                      None if drafted is None else _dense(drafted, "drafted", torch.int32, (M,), dev),
                      M, n, _dense(rows, "rows", torch.int32, (M, n), dev),
                      _dense(count, "count", torch.int32, (M,), dev), st)


# ---------------------------------------------------------------- pages given back and shared

def _lens_used(alloc: PageAllocator, lens_out, used_out):
    M, dev = alloc.members, alloc.device_index
    return (alloc.lens.data_ptr() if lens_out is None
            else _dense(lens_out, "lens_out", torch.int32, (M,), dev),
            alloc.used.data_ptr() if used_out is None
            else _dense(used_out, "used_out", torch.int32, (1,), dev))


def trim_pages(alloc: PageAllocator, new_lens: torch.Tensor, lens_out: torch.Tensor | None = None,
               used_out: torch.Tensor | None = None, stream=None) -> None:
    """Every member keeps its first new_lens[m] tokens (negative: out of use); the pages behind
    them that nobody else holds go back to the free list.  alloc.lens and alloc.used follow (or
    lens_out / used_out are written).  See ls_trim_pages for what is refused."""
    if stream is not None:
        with _as_current(stream):
            return trim_pages(alloc, new_lens, lens_out, used_out)
    M, dev = alloc.members, alloc.device_index
    st = _dev_stream(dev)
    lo, uo = _lens_used(alloc, lens_out, used_out)
    B.ls_trim_pages(alloc.block_table.data_ptr(), M, alloc.max_blocks, alloc.page_size,
                    alloc.num_pages, alloc.lens.data_ptr(),
                    _dense(new_lens, "new_lens", torch.int32, (M,), dev), alloc.free_list.data_ptr(),
                    alloc.num_free, alloc.used.data_ptr(),
                    None if alloc.shared is None else alloc.shared.data_ptr(), lo, uo, st)


def fork_pages(alloc: PageAllocator, src: torch.Tensor, keep: torch.Tensor | None = None,
               copies: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
               used_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Member m with src[m] >= 0 becomes a branch of that member's first keep[m] tokens (default:
    all).  Whole pages are shared; returns copies int32 [3][members], what copy_pages has to
    copy of the partial ones.  See ls_fork_pages for what is refused."""
    if stream is not None:
        with _as_current(stream):
            return fork_pages(alloc, src, keep, copies, lens_out, used_out)
    M, dev = alloc.members, alloc.device_index
    st = _dev_stream(dev)
    if alloc.shared is None:
        raise ValueError("the allocator does not share pages (PageAllocator's shared)")
    if copies is None:
        copies = torch.empty((3, M), dtype=torch.int32, device=alloc.block_table.device)
    lo, uo = _lens_used(alloc, lens_out, used_out)
    B.ls_fork_pages(alloc.block_table.data_ptr(), M, alloc.max_blocks, alloc.page_size,
                    alloc.num_pages, alloc.lens.data_ptr(), _dense(src, "src", torch.int32, (M,), dev),
                    None if keep is None else _dense(keep, "keep", torch.int32, (M,), dev),
                    alloc.free_list.data_ptr(), alloc.num_free, alloc.used.data_ptr(),
                    alloc.shared.data_ptr(), _dense(copies, "copies", torch.int32, (3, M), dev), lo,
                    uo, st)
    return copies


def copy_pages(pools: LayerPools, copies: torch.Tensor, stream=None) -> None:
    """copies int32 [3][count]: the first copies[2][i] rows of page copies[0][i] to page
    copies[1][i], in every layer; (-1, -1) where there is nothing to copy."""
    if stream is not None:
        with _as_current(stream):
            return copy_pages(pools, copies)
    dev = copies.get_device()
    st = _dev_stream(dev)
    if pools.device_indices - {dev}:
        raise ValueError("the pools are on another device")
    n = copies.shape[1] if copies.dim() == 2 else -1
    p = _dense(copies, "copies", torch.int32, (3, n), dev)
    B.ls_copy_pages(pools.struct, pools.layers, pools.layer_stride, n, p, p + 4 * n, p + 8 * n, st)


# ---------------------------------------------------------------- token statistics

def _logit_rows(t: torch.Tensor, name: str, dtype, shape, dev: int):
    """(address, row stride) of [T][V] rows, each dense."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, dtype, shape, dev)
    T, V = shape
    rs, es = t.stride()
    if T <= 1:
        rs = V
    if (V > 1 and es != 1) or rs < V:
        raise ValueError(f"{name}: rows must be contiguous and may not overlap")
    return t.data_ptr(), rs


def _logits(logits: torch.Tensor):
    if logits.dim() != 2:
        raise ValueError("logits must be [T][V]")
    if logits.dtype is not torch.bfloat16 and logits.dtype is not torch.float32:
        raise ValueError("logits must be bf16 or fp32")
    dev = logits.get_device()
    p, rs = _logit_rows(logits, "logits", logits.dtype, logits.shape, dev)
    return dev, *logits.shape, B.LS_BF16 if logits.dtype is torch.bfloat16 else B.LS_FP32, p, rs


def token_logp_fwd(logits: torch.Tensor, targets: torch.Tensor | None, temperature: float = 1.0,
                   top: int = 0, stream=None):
    """Log probabilities of the targets, entropies and the `top` likeliest tokens of the rows:
    logits [T][V] bf16 or fp32 (rows may be apart, as of a padded vocabulary), targets int32 [T]
    (-1: a padding row; None: no log probabilities).  Returns (logp, lse, entropy, top_logp
    [T][top], top_ids [T][top]); None where there is none.  See ls_token_logp_fwd."""
    if stream is not None:
        with _as_current(stream):
            return token_logp_fwd(logits, targets, temperature, top)
    dev, T, V, dt, p, rs = _logits(logits)
    st = _dev_stream(dev)
    tp = None if targets is None else _dense(targets, "targets", torch.int32, (T,), dev)
    lse = torch.empty(T, dtype=torch.float32, device=logits.device)
    entropy = torch.empty_like(lse)
    logp = top_logp = top_ids = gp = lp = ip = None
    if targets is not None:
        logp = torch.empty_like(lse)
        gp = logp.data_ptr()
    if top > 0:
        top_logp = torch.empty((T, top), dtype=torch.float32, device=logits.device)
        top_ids = torch.empty((T, top), dtype=torch.int32, device=logits.device)
        lp, ip = top_logp.data_ptr(), top_ids.data_ptr()
    if T > 0:
        _with_workspace(B.ls_token_logp_fwd,
                        (p, dt, T, V, rs, tp, temperature, top, gp, lse.data_ptr(),
                         entropy.data_ptr(), lp, ip),
                        lambda: B.ls_token_logp_fwd_workspace(dt, T, V, top), logits, "token_logp", st)
    return logp, lse, entropy, top_logp, top_ids


def token_logp_bwd(logits: torch.Tensor, targets: torch.Tensor | None, lse: torch.Tensor,
                   entropy: torch.Tensor | None, d_logp: torch.Tensor | None,
                   d_entropy: torch.Tensor | None = None, temperature: float = 1.0,
                   top_ids: torch.Tensor | None = None, d_top: torch.Tensor | None = None,
                   dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient that an objective of token_logp_fwd's outputs sends to the logits: d_logp,
    d_entropy fp32 [T] (each or None), d_top fp32 [T][top] with top_ids.  lse and entropy are
    the forward's; temperatures from 1e-3 on.  dlogits may be the logits themselves.  Returns
    dlogits."""
    if stream is not None:
        with _as_current(stream):
            return token_logp_bwd(logits, targets, lse, entropy, d_logp, d_entropy, temperature,
                                  top_ids, d_top, dlogits)
    dev, T, V, dt, p, rs = _logits(logits)
    st = _dev_stream(dev)

    def row(t, name, dtype=torch.float32):
        return None if t is None else _dense(t, name, dtype, (T,), dev)

    if dlogits is None:
        dlogits = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
    dp, drs = _logit_rows(dlogits, "dlogits", logits.dtype, logits.shape, dev)
    if (top_ids is None) != (d_top is None):
        raise ValueError("top_ids and d_top go together")
    top, ip, tp = 0, None, None
    if d_top is not None:
        top = d_top.shape[1] if d_top.dim() == 2 else -1
        ip = _dense(top_ids, "top_ids", torch.int32, (T, top), dev)
        tp = _dense(d_top, "d_top", torch.float32, (T, top), dev)
    B.ls_token_logp_bwd(p, dt, T, V, rs, row(targets, "targets", torch.int32), temperature,
                        row(lse, "lse"), row(entropy, "entropy"), top, ip, row(d_logp, "d_logp"),
                        row(d_entropy, "d_entropy"), tp, dp, drs, st)
    return dlogits
