"""Torch-facing wrappers over libtpa. Tensors are only allocated here and
their pointers handed to the library; no arithmetic of the method runs in
Python."""
from __future__ import annotations

import ctypes as C
from typing import Sequence

import numpy as np
import torch

from ._abi import (BALANCE_FFD, BALANCE_KK, GRAD_BF16, GRAD_F32, LOGITS_BF16, LOGITS_COMPACT, LOGITS_F32, LOGITS_PADDED,
                   MASK_BITS, MASK_U8, PAGED_POOL, PAGED_VIEW, ROPE_PARAMS, SAMPLE_PARAMS, WEIGHT_BF16, WEIGHT_F32,
                   BlockMaskView, PackingMetrics, TreeInfo, TreeView, check, lib)


def _stream_ptr(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


class Tree:
    """Packed trees on the host (owns a library tree handle)."""

    def __init__(self, handle: C.c_void_p):
        self._h = handle
        info = TreeInfo()
        check("tpa_tree_get_info", lib().tpa_tree_get_info(self._h, C.byref(info)))
        self.info = info

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            lib().tpa_tree_free(h)
            self._h = None

    @property
    def n_trees(self) -> int:
        return self.info.n_trees

    @property
    def t_pad(self) -> int:
        return self.info.t_pad

    @property
    def tree_token_ratio(self) -> float:
        return self.info.tree_token_ratio

    def host_view(self) -> TreeView:
        v = TreeView()
        base = lib().tpa_tree_host_blob(self._h)
        check("tpa_tree_make_view", lib().tpa_tree_make_view(self._h, base, C.byref(v)))
        return v

    def host_blob(self) -> np.ndarray:
        """A copy of the metadata blob (uint8)."""
        base = lib().tpa_tree_host_blob(self._h)
        return np.ctypeslib.as_array((C.c_uint8 * self.info.blob_bytes).from_address(base)).copy()

    def arrays(self) -> dict[str, np.ndarray]:
        """Copies of every metadata array, shaped per tree."""
        v = self.host_view()
        B, T, S, N, M = (self.info.n_trees, self.info.t_pad, self.info.n_seqs,
                         self.info.total_seq_tokens, self.info.max_nodes)

        def arr(ptr, ctype, n, shape):
            return np.ctypeslib.as_array((ctype * n).from_address(ptr)).reshape(shape).copy()

        return {
            "tokens": arr(v.tokens, C.c_int32, B * T, (B, T)),
            "subtree_end": arr(v.subtree_end, C.c_int32, B * T, (B, T)),
            "parent": arr(v.parent, C.c_int32, B * T, (B, T)),
            "depth": arr(v.depth, C.c_int32, B * T, (B, T)),
            "node_id": arr(v.node_id, C.c_int32, B * T, (B, T)),
            "child_off": arr(v.child_off, C.c_int32, B * (T + 1), (B, T + 1)),
            "child_pos": arr(v.child_pos, C.c_int32, B * T, (B, T)),
            "n_tokens": arr(v.n_tokens, C.c_int32, B, (B,)),
            "tok_base": arr(v.tok_base, C.c_int64, B + 1, (B + 1,)),
            "node_info": arr(v.node_info, C.c_int32, B * M * 4, (B, M, 4)),
            "n_nodes": arr(v.n_nodes, C.c_int32, B, (B,)),
            "seq_tree": arr(v.seq_tree, C.c_int32, S, (S,)),
            "seq_off": arr(v.seq_off, C.c_int64, S + 1, (S + 1,)),
            "seq_pos": arr(v.seq_pos, C.c_int32, N, (N,)),
        }

    def upload(self, device="cuda", stream=None, buffer: torch.Tensor | None = None) -> "DeviceTree":
        """Copy the metadata blob into device memory (a torch uint8 buffer)."""
        nbytes = int(self.info.blob_bytes)
        if buffer is None:
            buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        check("tpa_tree_upload", lib().tpa_tree_upload(self._h, buffer.data_ptr(), buffer.numel(),
                                                       _stream_ptr(stream)))
        return DeviceTree(self, buffer)


class DeviceTree:
    """Packed-tree metadata resident on the device."""

    def __init__(self, tree: Tree, buf: torch.Tensor):
        self.tree = tree
        self.buf = buf
        self.view = TreeView()
        check("tpa_tree_make_view", lib().tpa_tree_make_view(tree._h, buf.data_ptr(), C.byref(self.view)))

    @property
    def info(self) -> TreeInfo:
        return self.tree.info

    @property
    def device(self) -> torch.device:
        return self.buf.device


class BlockMask:
    """128x128 tile classes and the two CSR lists, in one device buffer."""

    def __init__(self, n_trees: int, t_pad: int, device, buf: torch.Tensor | None = None):
        nbytes = int(lib().tpa_blockmask_bytes(n_trees, t_pad))
        if buf is None:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.buf = buf
        self.view = BlockMaskView()
        check("tpa_blockmask_make_view",
              lib().tpa_blockmask_make_view(buf.data_ptr(), n_trees, t_pad, C.byref(self.view)))
        self.n_trees, self.t_pad, self.n_blk, self.cap = n_trees, t_pad, self.view.n_blk, self.view.cap

    def _slice(self, ptr: int, nbytes: int, dtype, shape):
        off = ptr - self.buf.data_ptr()
        return self.buf[off:off + nbytes].view(dtype).view(shape)

    def arrays(self) -> dict[str, torch.Tensor]:
        B, n, cap = self.n_trees, self.n_blk, self.cap
        v = self.view
        return {
            "cls": self._slice(v.cls, B * n * n, torch.uint8, (B, n, n)),
            "q_ptr": self._slice(v.q_ptr, 4 * B * (n + 1), torch.int32, (B, n + 1)),
            "q_idx": self._slice(v.q_idx, 4 * B * cap, torch.int32, (B, cap)),
            "k_ptr": self._slice(v.k_ptr, 4 * B * (n + 1), torch.int32, (B, n + 1)),
            "k_idx": self._slice(v.k_idx, 4 * B * cap, torch.int32, (B, cap)),
            "qmask": self._slice(v.qmask, 2048 * B * cap, torch.int32, (B, cap, 128, 4)),
            "sched": self._slice(v.sched, 4 * 16, torch.int32, (16,)),
        }


def tree_pack(seqs: Sequence[Sequence[int]] | None = None, max_tokens_per_mb: int = 8192, *,
              tokens: np.ndarray | None = None, offsets: np.ndarray | None = None) -> Tree:
    """Pack sequences (a list of token lists, or flat ``tokens`` + ``offsets``)."""
    if tokens is None:
        offsets = np.zeros(len(seqs) + 1, dtype=np.int64)
        offsets[1:] = np.cumsum([len(s) for s in seqs])
        tokens = np.fromiter((t for s in seqs for t in s), dtype=np.int32, count=int(offsets[-1]))
    tokens = np.ascontiguousarray(tokens, dtype=np.int32)
    offsets = np.ascontiguousarray(offsets, dtype=np.int64)
    h = C.c_void_p()
    n = len(offsets) - 1
    tok_p = tokens.ctypes.data_as(C.POINTER(C.c_int32)) if tokens.size else \
        C.cast(C.pointer(C.c_int32(0)), C.POINTER(C.c_int32))
    check("tpa_tree_pack", lib().tpa_tree_pack(tok_p, offsets.ctypes.data_as(C.POINTER(C.c_int64)), n,
                                               int(max_tokens_per_mb), C.byref(h)))
    return Tree(h)


def _padded(input_ids, attention_mask):
    ids = np.ascontiguousarray(np.asarray(input_ids), dtype=np.int32)
    msk = np.ascontiguousarray(np.asarray(attention_mask) != 0, dtype=np.uint8)
    if ids.ndim != 2 or ids.shape != msk.shape:
        raise ValueError("input_ids and attention_mask must be 2-D arrays of one shape")
    return ids, msk


def extract_sequences(input_ids, attention_mask) -> tuple[np.ndarray, np.ndarray]:
    """Real tokens of a padded batch (tpa_extract_sequences): flat int32
    tokens and int64 offsets, the input format of ``tree_pack``."""
    ids, msk = _padded(input_ids, attention_mask)
    n, L = ids.shape
    tokens = np.empty(n * L, dtype=np.int32)
    offsets = np.empty(n + 1, dtype=np.int64)
    check("tpa_extract_sequences", lib().tpa_extract_sequences(
        ids.ctypes.data_as(C.POINTER(C.c_int32)), msk.ctypes.data_as(C.POINTER(C.c_uint8)), n, L,
        tokens.ctypes.data_as(C.POINTER(C.c_int32)), offsets.ctypes.data_as(C.POINTER(C.c_int64))))
    return tokens[:int(offsets[-1])], offsets


def tree_pack_padded(input_ids, attention_mask, max_tokens_per_mb: int = 8192) -> Tree:
    """Extract the real tokens of a padded batch and pack them (tpa_tree_pack_padded)."""
    ids, msk = _padded(input_ids, attention_mask)
    h = C.c_void_p()
    check("tpa_tree_pack_padded", lib().tpa_tree_pack_padded(
        ids.ctypes.data_as(C.POINTER(C.c_int32)), msk.ctypes.data_as(C.POINTER(C.c_uint8)), ids.shape[0],
        ids.shape[1], int(max_tokens_per_mb), C.byref(h)))
    return Tree(h)


def balance(weights: Sequence[int], capacity: int, min_groups: int = 1, groups_divisor: int = 1,
            algorithm: str = "ffd") -> tuple[np.ndarray, int, str]:
    """Split weighted items into groups (tpa_balance): returns (group of each
    item, number of groups, algorithm whose result it is)."""
    w = np.ascontiguousarray(np.asarray(weights, dtype=np.int64))
    if algorithm not in ("ffd", "kk"):
        raise ValueError(f"unknown balancing algorithm {algorithm!r}; choose 'ffd' or 'kk'")
    algo = BALANCE_FFD if algorithm == "ffd" else BALANCE_KK
    out = np.empty(len(w), dtype=np.int32)
    ng, used = C.c_int32(0), C.c_int32(0)
    check("tpa_balance", lib().tpa_balance(w.ctypes.data_as(C.POINTER(C.c_int64)), len(w), int(capacity),
                                           int(min_groups), int(groups_divisor), algo,
                                           out.ctypes.data_as(C.POINTER(C.c_int32)), C.byref(ng),
                                           C.byref(used)))
    return out, ng.value, "kk" if used.value == BALANCE_KK else "ffd"


def packing_metrics(weights: Sequence[int], group_of: Sequence[int], n_groups: int, capacity: int) -> dict:
    """The packing metrics of a grouping (tpa_packing_metrics) as a dict."""
    w = np.ascontiguousarray(np.asarray(weights, dtype=np.int64))
    g = np.ascontiguousarray(np.asarray(group_of, dtype=np.int32))
    m = PackingMetrics()
    check("tpa_packing_metrics", lib().tpa_packing_metrics(w.ctypes.data_as(C.POINTER(C.c_int64)), len(w),
                                                           g.ctypes.data_as(C.POINTER(C.c_int32)), int(n_groups),
                                                           int(capacity), C.byref(m)))
    return {f: getattr(m, f) for f, _ in PackingMetrics._fields_ if f != "pad_"}


def dense_mask(dtree: DeviceTree, fmt: str = "u8", invert: bool = False, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Dense ancestor mask of every tree (tpa_dense_mask): uint8 [B, T, T]
    for fmt "u8", or int32 words [B, T, T/32] (bit j%32 of word j/32) for
    fmt "bits"; 1 marks a visible pair, or a removed pair with invert."""
    if fmt not in ("u8", "bits"):
        raise ValueError(f"unknown mask format {fmt!r}; choose 'u8' or 'bits'")
    B, T = dtree.info.n_trees, dtree.info.t_pad
    code = MASK_U8 if fmt == "u8" else MASK_BITS
    if out is None:
        out = (torch.empty((B, T, T), dtype=torch.uint8, device=dtree.device) if fmt == "u8" else
               torch.empty((B, T, T // 32), dtype=torch.int32, device=dtree.device))
    nbytes = out.numel() * out.element_size()
    check("tpa_dense_mask", lib().tpa_dense_mask(C.byref(dtree.view), out.data_ptr(), nbytes, code,
                                                 1 if invert else 0, _stream_ptr(stream)))
    return out


def block_classify(dtree: DeviceTree, stream=None, out: BlockMask | None = None) -> BlockMask:
    mask = out or BlockMask(dtree.info.n_trees, dtree.info.t_pad, dtree.device)
    check("tpa_block_classify", lib().tpa_block_classify(C.byref(dtree.view), C.byref(mask.view),
                                                         _stream_ptr(stream)))
    return mask


def _check_qkv(dtree: DeviceTree, q, k, v):
    B, T = dtree.info.n_trees, dtree.info.t_pad
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, T_pad, H, d]")
        if t.shape[0] != B or t.shape[1] != T:
            raise ValueError(f"{name} has shape {tuple(t.shape)}; expected [{B}, {T}, H, d]")
    if k.shape != v.shape or q.shape[3] != k.shape[3]:
        raise ValueError("k and v must match, and share head_dim with q")
    return B, T, q.shape[2], k.shape[2], q.shape[3]


def tree_attn_fwd(dtree: DeviceTree, mask: BlockMask, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  softmax_scale: float | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, stream=None):
    """Tree attention forward: returns O [B, T_pad, Hq, d] bf16 and LSE [B, Hq, T_pad] fp32."""
    B, T, Hq, Hkv, d = _check_qkv(dtree, q, k, v)
    o = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    check("tpa_tree_attn_fwd", lib().tpa_tree_attn_fwd(
        C.byref(dtree.view), C.byref(mask.view), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
        lse.data_ptr(), Hq, Hkv, d, float(softmax_scale or 0.0), _stream_ptr(stream)))
    return o, lse


_GRAD = {torch.float32: GRAD_F32, torch.bfloat16: GRAD_BF16}


def tree_attn_bwd_workspace_bytes(n_trees: int, t_pad: int, n_heads_q: int, n_heads_kv: int, head_dim: int,
                                  grad_dtype: torch.dtype = torch.float32) -> int:
    return int(lib().tpa_tree_attn_bwd_workspace_bytes(n_trees, t_pad, n_heads_q, n_heads_kv, head_dim,
                                                       _GRAD[grad_dtype]))


def tree_attn_bwd(dtree: DeviceTree, mask: BlockMask, q, k, v, o, lse, dout,
                  softmax_scale: float | None = None, workspace: torch.Tensor | None = None,
                  out: tuple | None = None, grad_dtype: torch.dtype = torch.float32, stream=None):
    """Tree attention backward: returns dQ, dK, dV shaped like q, k, v, in
    ``grad_dtype`` (fp32 by default, or bf16)."""
    B, T, Hq, Hkv, d = _check_qkv(dtree, q, k, v)
    if dout.shape != q.shape or dout.dtype != torch.bfloat16 or not dout.is_contiguous():
        raise ValueError("dout must be a contiguous bf16 tensor shaped like q")
    if grad_dtype not in _GRAD:
        raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
    if workspace is None:
        nbytes = tree_attn_bwd_workspace_bytes(B, T, Hq, Hkv, d, grad_dtype)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if out is None:
        out = tuple(torch.empty(x.shape, dtype=grad_dtype, device=x.device) for x in (q, k, v))
    dq, dk, dv = out
    if not all(x.dtype == grad_dtype and x.is_contiguous() for x in out):
        raise ValueError("gradient buffers must be contiguous and of grad_dtype")
    check("tpa_tree_attn_bwd", lib().tpa_tree_attn_bwd(
        C.byref(dtree.view), C.byref(mask.view), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
        lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
        workspace.numel(), Hq, Hkv, d, float(softmax_scale or 0.0), _GRAD[grad_dtype], _stream_ptr(stream)))
    return dq, dk, dv


def tree_logprobs_entropy(dtree: DeviceTree, logits: torch.Tensor, layout: str = "compact",
                          out: tuple | None = None, stream=None):
    """Per-position (pos_logp, pos_entropy: [B, T_pad]) and per-sequence
    (seq_logp, seq_entropy: [total_seq_tokens]) fp32 results."""
    if logits.dtype != torch.bfloat16 or logits.dim() != 2 or logits.stride(1) != 1 or not logits.is_cuda:
        raise ValueError("logits must be a CUDA bf16 [rows, V] tensor with unit column stride")
    lay = {"compact": LOGITS_COMPACT, "padded": LOGITS_PADDED}[layout]
    B, T, N = dtree.info.n_trees, dtree.info.t_pad, dtree.info.total_seq_tokens
    dev = logits.device
    if out is None:
        out = (torch.empty((B, T), dtype=torch.float32, device=dev), torch.empty((B, T), dtype=torch.float32, device=dev),
               torch.empty(N, dtype=torch.float32, device=dev), torch.empty(N, dtype=torch.float32, device=dev))
    pl, pe, sl, se = out
    check("tpa_tree_logprobs_entropy", lib().tpa_tree_logprobs_entropy(
        C.byref(dtree.view), logits.data_ptr(), logits.stride(0), lay, logits.shape[1], pl.data_ptr(),
        pe.data_ptr(), sl.data_ptr(), se.data_ptr(), _stream_ptr(stream)))
    return pl, pe, sl, se


def lm_head_workspace_bytes(rows: int, vocab: int, n_trees: int, t_pad: int) -> int:
    return int(lib().tpa_lm_head_workspace_bytes(int(rows), int(vocab), int(n_trees), int(t_pad)))


def lm_head_logprobs_entropy(dtree: DeviceTree, hidden: torch.Tensor, weight: torch.Tensor,
                             out: tuple | None = None, workspace: torch.Tensor | None = None, stream=None):
    """The log-prob pass with the LM head fused in: ``hidden`` [tree tokens, H]
    (compact rows) and ``weight`` [V, H], both CUDA bf16; returns the four
    outputs of ``tree_logprobs_entropy`` without forming the logits."""
    for name, t in (("hidden", hidden), ("weight", weight)):
        if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous CUDA bf16 matrix")
    if hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden and weight must have the same hidden size")
    B, T, N = dtree.info.n_trees, dtree.info.t_pad, dtree.info.total_seq_tokens
    rows, V, H = hidden.shape[0], weight.shape[0], hidden.shape[1]
    if rows != dtree.info.total_tree_tokens:
        raise ValueError("hidden must have one row per tree token (compact rows)")
    dev = hidden.device
    if out is None:
        out = (torch.empty((B, T), dtype=torch.float32, device=dev), torch.empty((B, T), dtype=torch.float32, device=dev),
               torch.empty(N, dtype=torch.float32, device=dev), torch.empty(N, dtype=torch.float32, device=dev))
    nbytes = lm_head_workspace_bytes(rows, V, B, T)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    pl, pe, sl, se = out
    check("tpa_lm_head_logprobs_entropy", lib().tpa_lm_head_logprobs_entropy(
        C.byref(dtree.view), hidden.data_ptr(), weight.data_ptr(), H, V, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), pl.data_ptr(), pe.data_ptr(), sl.data_ptr(), se.data_ptr(),
        _stream_ptr(stream)))
    return pl, pe, sl, se


def _launch_stream(stream, first: torch.Tensor, *tensors) -> int:
    """The stream of a call, after a check that its tensors (None is passed
    over) are on the one CUDA device that is current: the library launches there."""
    dev = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("every tensor must be a CUDA tensor, all on one device")
    if dev < 0:
        raise ValueError("every tensor must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_ptr(stream)


def _new(stream, shape, dtype: torch.dtype, device) -> torch.Tensor:
    """Uninitialised memory of the stream that the call runs on: what the
    current one still has under way cannot reach it, and it is used again, once
    dropped, behind the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(st):
        return torch.empty(shape, dtype=dtype, device=device)


def _int32(name: str, value) -> int:
    """A whole number that the library takes in 32 bits (ctypes would cut off the others)."""
    n = int(value)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits")
    return n


def _whole_workspace(workspace) -> None:
    """A workspace's size is counted from its elements: each has to have memory of its own, behind the one before."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _head_rows(name: str, t: torch.Tensor, dtypes=(torch.bfloat16,)) -> tuple[int, int, int, int]:
    """(rows, row stride, heads, d) of a tensor [..., H, d] whose heads are
    contiguous and whose leading dimensions are evenly spaced rows."""
    if t.dim() == 3 and t.dtype in dtypes:
        (n, H, d), (row, head, one) = t.shape, t.stride()
        if one == 1 and (head == d or H == 1):
            return n, (row if n > 1 else H * d), H, d
    if t.dtype not in dtypes or t.dim() < 3:
        raise ValueError(f"{name} must be [..., heads, d] of {' or '.join(str(x) for x in dtypes)}")
    H, d = t.shape[-2:]
    if t.stride(-1) != 1 or (H > 1 and t.stride(-2) != d):
        raise ValueError(f"{name} must have its heads and their values contiguous")
    rows, stride = t.shape[-3], t.stride(-3)
    if rows == 1:
        stride = H * d
    for i in range(t.dim() - 4, -1, -1):
        if t.shape[i] != 1:
            if rows == 1:
                stride = t.stride(i)
            elif t.stride(i) != rows * stride:
                raise ValueError(f"the leading dimensions of {name} must be evenly spaced rows")
            rows *= t.shape[i]
    return rows, stride, H, d


def rope_table(n_positions: int, rot_dim: int, base: float = 10000.0, inv_freq: Sequence[float] | None = None,
               scale: float = 1.0, device="cuda", out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Cosines and sines of the rotary positions (tpa_rope_table): fp32
    [n_positions, rot_dim], cos | sin, made once for a model.  ``inv_freq``
    gives the rot_dim / 2 frequencies in place of ``base`` ** (-2 j / rot_dim)."""
    fr = None
    n_positions, rot_dim = _int32("n_positions", n_positions), _int32("rot_dim", rot_dim)
    if inv_freq is not None:
        if len(inv_freq) != rot_dim // 2:
            raise ValueError("inv_freq must hold rot_dim / 2 frequencies")
        fr = (C.c_double * len(inv_freq))(*[float(f) for f in inv_freq])
    if out is None:
        out = _new(stream, (n_positions, rot_dim), torch.float32, device)
    if out.dtype != torch.float32 or not out.is_contiguous() or tuple(out.shape) != (n_positions, rot_dim):
        raise ValueError("out must be a contiguous fp32 tensor [n_positions, rot_dim]")
    st = _launch_stream(stream, out)
    check("tpa_rope_table", lib().tpa_rope_table(out.data_ptr(), n_positions, rot_dim, float(base), fr, float(scale),
                                                 st))
    return out


def _rope_params(table, q_weight, k_weight, eps, interleaved, d) -> bytes:
    """A tpa_rope_params as bytes (a ctypes structure takes longer to fill than the kernel to launch)."""
    at = rows = rot = wt = wq = wk = 0
    if table is not None:
        if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous fp32 tensor [positions, rot_dim]")
        at = table.data_ptr()
        rows, rot = table.shape
    if (q_weight is None) != (k_weight is None):
        raise ValueError("give both norm weights or neither")
    if q_weight is not None:
        dt = q_weight.dtype
        if (dt not in _WEIGHT or k_weight.dtype != dt or q_weight.numel() != d or k_weight.numel() != d or
                not q_weight.is_contiguous() or not k_weight.is_contiguous()):
            raise ValueError("norm weights must be contiguous, of d values, both fp32 or both bf16")
        wt, wq, wk = _WEIGHT[dt], q_weight.data_ptr(), k_weight.data_ptr()
    return ROPE_PARAMS.pack(at, rows, rot, 1 if interleaved else 0, wt, wq, wk, eps, 0)


_WEIGHT = {torch.float32: WEIGHT_F32, torch.bfloat16: WEIGHT_BF16}


def _positions(positions, rows: int):
    """(positions pointer, n_tokens pointer, t_pad, device) of an int32 tensor or a packed tree."""
    if isinstance(positions, DeviceTree):
        v = positions.view
        if rows != v.n_trees * v.t_pad:
            raise ValueError(f"q has {rows} rows; the tree has {v.n_trees} x {v.t_pad} positions")
        return v.depth, v.n_tokens, v.t_pad, positions.buf
    if positions.dtype != torch.int32 or not positions.is_contiguous() or positions.numel() != rows:
        raise ValueError("positions must be a contiguous int32 tensor with one entry a row of q, or a DeviceTree")
    return positions.data_ptr(), None, 0, positions


def qk_norm_rope_fwd(positions: "torch.Tensor | DeviceTree", q: torch.Tensor, k: torch.Tensor, table: torch.Tensor,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, out: tuple | None = None, stream=None):
    """RMS norm of every query and key head (with weights) and rotation by
    position in one pass (tpa_qk_norm_rope_fwd): returns q and k, bf16.

    q [..., Hq, d] and k [..., Hkv, d] bf16 may be slices of a fused
    projection; ``positions`` is an int32 tensor of their rows (negative:
    padding, which comes out 0) or a ``DeviceTree`` (token depths; q and k then
    are [B, T_pad, H, d] and the results go to ``tree_attn_fwd``)."""
    rows, sq, Hq, d = _head_rows("q", q)
    rows_k, sk, Hkv, dk = _head_rows("k", k)
    if rows_k != rows or dk != d:
        raise ValueError("q and k must have the same rows and head_dim")
    pos, n_tok, t_pad, pbuf = _positions(positions, rows)
    rp = _rope_params(table, q_weight, k_weight, eps, interleaved, d)
    st = _launch_stream(stream, q, k, table, q_weight, k_weight, pbuf, *(out or ()))
    if out is None:
        qo, ko = _new(stream, q.shape, q.dtype, q.device), _new(stream, k.shape, k.dtype, k.device)
        so, sko = Hq * d, Hkv * d
    else:
        qo, ko = out
        if qo.shape != q.shape or ko.shape != k.shape:
            raise ValueError("out must be shaped like q and k")
        so, sko = _head_rows("out[0]", qo)[1], _head_rows("out[1]", ko)[1]
    check("tpa_qk_norm_rope_fwd", lib().tpa_qk_norm_rope_fwd(
        pos, n_tok, t_pad, rows, q.data_ptr(), sq, k.data_ptr(), sk, rp, qo.data_ptr(), so, ko.data_ptr(), sko, Hq,
        Hkv, d, st))
    return qo, ko


def qk_norm_rope_bwd(positions: "torch.Tensor | DeviceTree", dq_out: torch.Tensor, dk_out: torch.Tensor,
                     q: torch.Tensor | None, k: torch.Tensor | None, table: torch.Tensor,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, grad_dtype: torch.dtype = torch.bfloat16, out: tuple | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Gradients of ``qk_norm_rope_fwd`` (tpa_qk_norm_rope_bwd): from those of
    its outputs (fp32 or bf16, as ``tree_attn_bwd`` returns them) and its inputs
    q, k (needed with weights only) returns dq, dk of ``grad_dtype`` and the
    weights' gradients, fp32 (None without weights)."""
    if grad_dtype not in _GRAD or dq_out.dtype != dk_out.dtype:
        raise ValueError("gradients must be fp32 or bf16, dq_out and dk_out alike")
    rows, sgq, Hq, d = _head_rows("dq_out", dq_out, _GRAD)
    rows_k, sgk, Hkv, dk_ = _head_rows("dk_out", dk_out, _GRAD)
    if rows_k != rows or dk_ != d:
        raise ValueError("dq_out and dk_out must have the same rows and head_dim")
    pos, n_tok, t_pad, pbuf = _positions(positions, rows)
    rp = _rope_params(table, q_weight, k_weight, eps, interleaved, d)
    norm = q_weight is not None
    sq = sk = 0
    if norm:
        if q is None or k is None or q.shape != dq_out.shape or k.shape != dk_out.shape:
            raise ValueError("q and k must be given with the weights, shaped like dq_out and dk_out")
        sq, sk = _head_rows("q", q)[1], _head_rows("k", k)[1]
    _whole_workspace(workspace)
    dev = dq_out.device
    st = _launch_stream(stream, dq_out, dk_out, table, q_weight, k_weight, pbuf, workspace, *(out or ()),
                        *((q, k) if norm else ()))
    if out is None:
        dq, dk = _new(stream, dq_out.shape, grad_dtype, dev), _new(stream, dk_out.shape, grad_dtype, dev)
        so, sko = Hq * d, Hkv * d
    else:
        dq, dk = out
        if dq.shape != dq_out.shape or dk.shape != dk_out.shape or dq.dtype != grad_dtype or dk.dtype != grad_dtype:
            raise ValueError("out must be shaped like dq_out and dk_out and of grad_dtype")
        so, sko = _head_rows("out[0]", dq, _GRAD)[1], _head_rows("out[1]", dk, _GRAD)[1]
    dwq = dwk = None
    if norm:
        dwq, dwk = (_new(stream, d, torch.float32, dev) for _ in range(2))
        if workspace is None:
            workspace = _new(stream, int(lib().tpa_qk_norm_rope_bwd_workspace_bytes(d)), torch.uint8, dev)
    check("tpa_qk_norm_rope_bwd", lib().tpa_qk_norm_rope_bwd(
        pos, n_tok, t_pad, rows, dq_out.data_ptr(), sgq, dk_out.data_ptr(), sgk, _GRAD[dq_out.dtype],
        q.data_ptr() if norm else None, sq, k.data_ptr() if norm else None, sk, rp, dq.data_ptr(), so,
        dk.data_ptr(), sko, _GRAD[grad_dtype], _ptr(dwq), _ptr(dwk), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), Hq, Hkv, d, st))
    return dq, dk, dwq, dwk


def _paged_view(k_cache, v_cache, pages, offsets, kv_lens, n_rows: int, n_heads_kv: int | None, d: int):
    """A tpa_paged_view as bytes, and the cache's key/value heads."""
    bf16, i32 = torch.bfloat16, torch.int32
    shape = k_cache.shape
    if (k_cache.dtype != bf16 or v_cache.dtype != bf16 or len(shape) != 4 or not k_cache.is_contiguous() or
            not v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous bf16 tensors [n_pages, Hkv, page_size, d]")
    n_pages, hkv, page, dc = shape
    if v_cache.shape != shape or dc != d or (n_heads_kv is not None and n_heads_kv != hkv):
        raise ValueError("k_cache and v_cache must match, and have the head_dim and key/value heads of the new tokens")
    if pages.dtype != i32 or pages.dim() != 2 or pages.stride(1) != 1:
        raise ValueError("pages must be an int32 tensor [n_seqs, max_pages] with unit column stride")
    n, width = pages.shape
    if (offsets.dtype != i32 or kv_lens.dtype != i32 or offsets.shape != (n + 1,) or kv_lens.shape != (n,) or
            not offsets.is_contiguous() or not kv_lens.is_contiguous()):
        raise ValueError("offsets [n_seqs + 1] and kv_lens [n_seqs] must be contiguous int32 tensors")
    return PAGED_VIEW.pack(k_cache.data_ptr(), v_cache.data_ptr(), pages.data_ptr(), offsets.data_ptr(),
                           kv_lens.data_ptr(), n_pages, page, n, width, pages.stride(0) if n > 1 else max(width, 1),
                           hkv, d, n_rows), hkv


def paged_append(k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor, offsets: torch.Tensor,
                 kv_lens: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
                 table: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Write the new tokens' keys (normed with weights, rotated with a table)
    and values into a paged cache (tpa_paged_append); with ``q`` also returns
    the queries, normed and rotated, for ``paged_attn_fwd``.

    Caches are bf16 [n_pages, Hkv, page_size, d]; ``pages`` [n_seqs, max_pages],
    ``offsets`` [n_seqs + 1] and ``kv_lens`` [n_seqs] (the new tokens included)
    are int32 device tensors; q, k, v are [tokens, H, d], rows behind
    offsets[n_seqs] padding (their rows of the result are not written)."""
    rows, sk, Hkv, d = _head_rows("k", k)
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    sv = _head_rows("v", v)[1]
    cache, _ = _paged_view(k_cache, v_cache, pages, offsets, kv_lens, rows, Hkv, d)
    rp = _rope_params(table, q_weight, k_weight, eps, interleaved, d)
    sq = so = Hq = 0
    if q is not None:
        rows_q, sq, Hq, dq = _head_rows("q", q)
        if rows_q != rows or dq != d:
            raise ValueError("q must have the rows and head_dim of k")
        so = Hq * d
        if q_out is not None:
            if q_out.shape != q.shape:
                raise ValueError("q_out must be shaped like q")
            so = _head_rows("q_out", q_out)[1]
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _launch_stream(stream, k, v, q, q_out, k_cache, v_cache, pages, offsets, kv_lens, table, q_weight, k_weight)
    if q is not None and q_out is None:
        q_out = _new(stream, q.shape, q.dtype, q.device)
    check("tpa_paged_append", lib().tpa_paged_append(cache, k.data_ptr(), sk, v.data_ptr(), sv, _ptr(q), sq,
                                                     _ptr(q_out), so, Hq, rp, st))
    return q_out


def paged_attn_workspace_bytes(max_q_len: int, n_heads_q: int, n_heads_kv: int, head_dim: int) -> int:
    return int(lib().tpa_paged_attn_workspace_bytes(
        _int32("max_q_len", max_q_len), _int32("n_heads_q", n_heads_q), _int32("n_heads_kv", n_heads_kv),
        _int32("head_dim", head_dim)))


def paged_attn_fwd(k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor, offsets: torch.Tensor,
                   kv_lens: torch.Tensor, q: torch.Tensor, max_q_len: int, softmax_scale: float | None = None,
                   window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """Attention of each sequence's new tokens over its pages, causal at the
    sequence's end (tpa_paged_attn_fwd): returns O [tokens, Hq, d] bf16 and LSE
    [tokens, Hq] fp32.

    The batch is described as for ``paged_append``, which is called first (its
    result is ``q``); ``max_q_len`` is the most new tokens of any sequence and
    ``window`` limits each token to that many keys (0: all)."""
    return _paged_attend(k_cache, v_cache, pages, offsets, kv_lens, q, None, None, max_q_len, softmax_scale, window, out, lse,
                         workspace, stream)


def paged_attn_tree_fwd(k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor, offsets: torch.Tensor,
                        kv_lens: torch.Tensor, q: torch.Tensor, masks: torch.Tensor, max_q_len: int,
                        positions: torch.Tensor | None = None, softmax_scale: float | None = None, window: int = 0,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """``paged_attn_fwd`` for drafted trees (tpa_paged_attn_tree_fwd): a new token
    sees what its sequence has cached before the new ones, and of those the ones
    whose bits its row of ``masks`` [tokens, words] int32 has set.

    ``draft_masks`` makes the masks from a tree's parents (once a step, for all
    layers), and the ``positions`` that are needed with a ``window``; give it the same window.
    The workspace is ``paged_attn_fwd``'s."""
    if masks.dtype != torch.int32 or masks.dim() != 2 or masks.shape[0] != q.shape[0] or not masks.is_contiguous():
        raise ValueError("masks must be a contiguous int32 tensor [tokens, words]")
    if not 1 <= masks.shape[1] <= 32:
        raise ValueError("masks must have 1 to 32 words a row")
    if positions is not None and (positions.dtype != torch.int32 or positions.shape != q.shape[:1] or
                                  not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 tensor [tokens]")
    if positions is None and window:
        raise ValueError("a window needs the tokens' positions")
    return _paged_attend(k_cache, v_cache, pages, offsets, kv_lens, q, masks, positions, max_q_len, softmax_scale, window, out,
                         lse, workspace, stream)


def _paged_attend(k_cache, v_cache, pages, offsets, kv_lens, q, masks, positions, max_q_len, softmax_scale, window, out, lse,
                  workspace, stream):
    rows, sq, Hq, d = _head_rows("q", q)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, Hq, d]")
    max_q_len, window = _int32("max_q_len", max_q_len), int(window)
    if window < 0:
        raise ValueError("window must not be negative")
    window = min(window, 2 ** 31 - 1)  # longer than any sequence
    cache, hkv = _paged_view(k_cache, v_cache, pages, offsets, kv_lens, rows, None, d)
    _whole_workspace(workspace)
    st = _launch_stream(stream, q, out, lse, workspace, k_cache, v_cache, pages, offsets, kv_lens, masks, positions)
    if out is None:
        o = _new(stream, q.shape, q.dtype, q.device)
    else:
        o = out
        if o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous():
            raise ValueError("out must be contiguous bf16 shaped like q")
    if lse is None:
        lse = _new(stream, (rows, Hq), torch.float32, q.device)
    elif lse.shape != (rows, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [tokens, Hq]")
    if workspace is None:
        workspace = _new(stream, paged_attn_workspace_bytes(max_q_len, Hq, hkv, d), torch.uint8, q.device)
    rest = (o.data_ptr(), lse.data_ptr(), Hq, max_q_len, float(softmax_scale or 0.0), window, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), st)
    if masks is None:
        check("tpa_paged_attn_fwd", lib().tpa_paged_attn_fwd(cache, q.data_ptr(), sq, *rest))
    else:
        check("tpa_paged_attn_tree_fwd", lib().tpa_paged_attn_tree_fwd(
            cache, q.data_ptr(), sq, masks.data_ptr(), masks.shape[1], _ptr(positions), *rest))
    return o, lse


def verify_drafts(target_probs: torch.Tensor, draft_tokens: torch.Tensor, u_accept: torch.Tensor,
                  u_next: torch.Tensor, draft_probs: torch.Tensor | None = None,
                  n_drafts: torch.Tensor | None = None, out: tuple | None = None, stream=None):
    """Accept or reject drafted tokens against the policy's probabilities and
    draw the next token, from given uniform numbers (tpa_verify_drafts).

    target_probs [S, K+1, V] and draft_probs [S, K, V] fp32 (None: drafts
    without probabilities), draft_tokens [S, K] int32, n_drafts [S] int32 (None:
    K each), u_accept [S, K] and u_next [S] fp32 in [0, 1).  Returns tokens
    [S, K+1] int32 (the accepted drafts, the drawn token, then -1) and the
    number accepted [S] int32."""
    if target_probs.dim() != 3 or draft_tokens.dim() != 2:
        raise ValueError("target_probs must be [S, K+1, V] and draft_tokens [S, K]")
    S, K1, V = target_probs.shape
    K = K1 - 1
    for name, n in (("the number of sequences", S), ("the number of drafts", K), ("the vocabulary", V)):
        _int32(name, n)
    i32, f32 = torch.int32, torch.float32
    if draft_tokens.dtype != i32 or draft_tokens.shape != (S, K) or not draft_tokens.is_contiguous():
        raise ValueError("draft_tokens must be a contiguous int32 tensor [S, K]")
    if (u_accept.dtype != f32 or u_accept.shape != (S, K) or not u_accept.is_contiguous() or u_next.dtype != f32 or
            u_next.shape != (S,) or not u_next.is_contiguous()):
        raise ValueError("u_accept [S, K] and u_next [S] must be contiguous fp32 tensors")
    if n_drafts is not None and (n_drafts.dtype != i32 or n_drafts.shape != (S,) or not n_drafts.is_contiguous()):
        raise ValueError("n_drafts must be a contiguous int32 tensor [S]")
    ts, tr, t1 = target_probs.stride()
    if target_probs.dtype != f32 or (V > 1 and t1 != 1) or (K > 0 and tr != V):
        raise ValueError("target_probs must be fp32 with contiguous sequences")
    ds = 0
    if draft_probs is not None:
        if draft_probs.dtype != f32 or draft_probs.shape != (S, K, V):
            raise ValueError("draft_probs must be fp32 [S, K, V]")
        ds, dr, d1 = draft_probs.stride()
        if (V > 1 and d1 != 1) or (K > 1 and dr != V):
            raise ValueError("draft_probs must have contiguous sequences")
    st = _launch_stream(stream, target_probs, draft_tokens, u_accept, u_next, draft_probs, n_drafts, *(out or ()))
    if out is None:
        dev = target_probs.device
        tokens, n_accepted = _new(stream, (S, K1), i32, dev), _new(stream, S, i32, dev)
    else:
        tokens, n_accepted = out
        if (tokens.dtype != i32 or tokens.shape != (S, K1) or not tokens.is_contiguous() or
                n_accepted.dtype != i32 or n_accepted.shape != (S,) or not n_accepted.is_contiguous()):
            raise ValueError("out must be contiguous int32 tensors [S, K+1] and [S]")
    if S == 1:
        ts, ds = K1 * V, K * V
    check("tpa_verify_drafts", lib().tpa_verify_drafts(
        target_probs.data_ptr(), ts, _ptr(draft_probs) if K else None, ds, draft_tokens.data_ptr(), _ptr(n_drafts),
        u_accept.data_ptr(), u_next.data_ptr(), tokens.data_ptr(), n_accepted.data_ptr(), S, K, V, st))
    return tokens, n_accepted


_I32 = torch.int32


def _vector(name: str, t: torch.Tensor, n: int) -> int:
    """The address of a contiguous int32 tensor [n]."""
    if t.dtype is _I32 and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous int32 tensor [{n}]")


def _table(name: str, t: torch.Tensor, n: int, m: int) -> int:
    """The address of a contiguous int32 tensor [n, m]."""
    if t.dtype is _I32 and t.shape == (n, m) and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous int32 tensor [{n}, {m}]")


def draft_masks(parents: torch.Tensor, offsets: torch.Tensor, kv_lens: torch.Tensor, max_q_len: int, window: int = 0,
                out: tuple | None = None, stream=None):
    """Positions [tokens] and masks [tokens, ceil(max_q_len / 32)], int32, of a
    batch's drafted trees (tpa_draft_masks): for ``qk_norm_rope_fwd`` and
    ``paged_attn_tree_fwd`` of a step's layers.

    ``parents`` [tokens] int32 has each new token's parent, its number among its
    sequence's new tokens (lower than its own), or -1 behind the last cached token;
    ``offsets`` and ``kv_lens`` are ``paged_append``'s, ``max_q_len`` <= 1024 the most new tokens of any sequence."""
    rows, n = parents.shape[0], kv_lens.shape[0]
    at = _vector("parents", parents, rows), _vector("offsets", offsets, n + 1), _vector("kv_lens", kv_lens, n)
    words, window = (int(max_q_len) + 31) // 32, int(window)
    if not 1 <= words <= 32 or window < 0:
        raise ValueError("max_q_len must be in [1, 1024] and window not negative")
    if out is None:
        st = _launch_stream(stream, parents, offsets, kv_lens)
        dev = parents.device
        positions, masks = _new(stream, (rows,), _I32, dev), _new(stream, (rows, words), _I32, dev)
    else:
        positions, masks = out
        _vector("positions", positions, rows)
        _table("masks", masks, rows, words)
        st = _launch_stream(stream, parents, offsets, kv_lens, positions, masks)
    check("tpa_draft_masks", lib().tpa_draft_masks(*at, n, rows, min(window, 2 ** 31 - 1), positions.data_ptr(),
                                                   masks.data_ptr(), words, st))
    return positions, masks


def accept_drafts(parents: torch.Tensor, offsets: torch.Tensor, draft_tokens: torch.Tensor, sampled: torch.Tensor,
                  max_path: int, out: tuple | None = None, stream=None):
    """The path that sampled tokens follow through drafted trees (tpa_accept_drafts).

    Row 0 of a sequence's new tokens is its last sampled token; behind a row that stands, its child stands whose
    ``draft_tokens`` entry is the one ``sampled`` behind the row (both [tokens] int32).  Returns tokens [S, max_path]
    (the sequences' next tokens, then -1), path [S, max_path] (the standing rows, then -1: for ``paged_compact``)
    and the number of standing rows [S], int32."""
    rows, n, most = parents.shape[0], offsets.shape[0] - 1, int(max_path)
    if not 1 <= most <= 1024:
        raise ValueError("max_path must be in [1, 1024]")
    at = (_vector("parents", parents, rows), _vector("offsets", offsets, n + 1), _vector("draft_tokens", draft_tokens, rows),
          _vector("sampled", sampled, rows))
    if out is None:
        st = _launch_stream(stream, parents, offsets, draft_tokens, sampled)
        dev = parents.device
        tokens, path, n_accepted = _new(stream, (n, most), _I32, dev), _new(stream, (n, most), _I32, dev), _new(stream, (n,), _I32, dev)
    else:
        tokens, path, n_accepted = out
        _table("tokens", tokens, n, most)
        _table("path", path, n, most)
        _vector("n_accepted", n_accepted, n)
        st = _launch_stream(stream, parents, offsets, draft_tokens, sampled, tokens, path, n_accepted)
    check("tpa_accept_drafts", lib().tpa_accept_drafts(*at, n, rows, tokens.data_ptr(), path.data_ptr(), n_accepted.data_ptr(),
                                                       most, st))
    return tokens, path, n_accepted


def _layers(k_cache, v_cache) -> tuple:
    """(layers, n_pages, Hkv, page_size, d) of bf16 caches of that shape, or of one layer's."""
    shape = k_cache.shape
    if (k_cache.dtype is not torch.bfloat16 or v_cache.dtype is not torch.bfloat16 or v_cache.shape != shape or
            not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous bf16 tensors of one shape")
    if len(shape) == 4:
        return (1, *shape)
    if len(shape) != 5 or shape[0] < 1:
        raise ValueError("k_cache and v_cache must be [layers, n_pages, Hkv, page_size, d] or one layer's")
    return tuple(shape)


def _pages(pages) -> tuple[int, int, int, int]:
    """(address, rows, width, row stride) of a page table."""
    if pages.dtype is not torch.int32 or pages.dim() != 2 or pages.stride(1) != 1:
        raise ValueError("pages must be an int32 tensor [n_seqs, max_pages] with unit column stride")
    n, width = pages.shape
    return pages.data_ptr(), n, width, pages.stride(0) if n > 1 else max(width, 1)


def paged_compact(k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor, offsets: torch.Tensor,
                  kv_lens: torch.Tensor, path: torch.Tensor, n_accepted: torch.Tensor, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Move an accepted path's keys and values to where their sequences go on
    (tpa_paged_compact), in all layers of caches [layers, n_pages, Hkv, page_size, d] (or one layer's); returns
    the sequences' new lengths [S] int32, ``kv_lens`` without the new tokens that do not stand.

    ``offsets`` and ``kv_lens`` are those of the step's ``paged_append``; ``path`` and ``n_accepted``
    come from ``accept_drafts``."""
    layers, n_pages, heads, page, d = _layers(k_cache, v_cache)
    at, n, width, stride = _pages(pages)
    if path.dim() != 2:
        raise ValueError("path must be an int32 tensor [n_seqs, max_path]")
    most = path.shape[1]
    # (the rows of the step's tensors are told by the offsets alone: no call has more)
    cache = PAGED_VIEW.pack(k_cache.data_ptr(), v_cache.data_ptr(), at, _vector("offsets", offsets, n + 1),
                            _vector("kv_lens", kv_lens, n), n_pages, page, n, width, stride, heads, d, 2 ** 30 - 1 if n else 0)
    at_path, at_n = _table("path", path, n, most), _vector("n_accepted", n_accepted, n)
    st = _launch_stream(stream, k_cache, v_cache, pages, offsets, kv_lens, path, n_accepted, out)
    if out is None:
        out = _new(stream, (n,), _I32, kv_lens.device)
    else:
        _vector("out", out, n)
    check("tpa_paged_compact", lib().tpa_paged_compact(cache, layers, at_path, at_n, most, out.data_ptr(), st))
    return out


def paged_resize(pages: torch.Tensor, kv_lens: torch.Tensor, refs: torch.Tensor, page_size: int,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Give every sequence the pages that its length needs (tpa_paged_resize):
    new ones for those that grow, none for those of length 0, whose pages go back.

    ``pages`` [S, max_pages] int32 (-1 where a row has no page) and ``refs`` [n_pages] int32 (0: free), both changed
    in place, are the state of a cache's pages: start with -1 and 0.  ``kv_lens`` [S] int32 are the lengths wanted.
    Returns the number of free pages left [1] int32; negative, and no row has grown, where that many are missing."""
    at, n, width, stride = _pages(pages)
    n_pages = refs.shape[0]
    pool = PAGED_POOL.pack(0, 0, at, _vector("kv_lens", kv_lens, n), _vector("refs", refs, n_pages), 0, n_pages,
                           _int32("page_size", page_size), 0, 0, n, width, stride)
    st = _launch_stream(stream, refs, pages, kv_lens, out)
    if out is None:
        out = _new(stream, (1,), _I32, refs.device)
    else:
        _vector("out", out, 1)
    check("tpa_paged_resize", lib().tpa_paged_resize(pool, out.data_ptr(), st))
    return out


def paged_fork(k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor, kv_lens: torch.Tensor,
               refs: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Make sequences copies of others (tpa_paged_fork), as the samples of a
    prompt are: rows ``dst`` [F] of ``pages`` and ``kv_lens`` become those of rows ``src`` [F], with whole
    pages shared and the last, partly filled one copied in all layers of the caches.

    State, caches and result as for ``paged_resize`` and ``paged_compact``; what the dst rows held goes back first."""
    layers, n_pages, heads, page, d = _layers(k_cache, v_cache)
    at, n, width, stride = _pages(pages)
    pool = PAGED_POOL.pack(k_cache.data_ptr(), v_cache.data_ptr(), at, _vector("kv_lens", kv_lens, n),
                           _vector("refs", refs, n_pages), layers, n_pages, page, heads, d, n, width, stride)
    forks = src.shape[0]
    at_src, at_dst = _vector("src", src, forks), _vector("dst", dst, forks)
    st = _launch_stream(stream, refs, k_cache, v_cache, pages, kv_lens, src, dst, out)
    if out is None:
        out = _new(stream, (1,), _I32, refs.device)
    else:
        _vector("out", out, 1)
    check("tpa_paged_fork", lib().tpa_paged_fork(pool, at_src, at_dst, forks, out.data_ptr(), st))
    return out


def _row_parameter(name: str, value: torch.Tensor, rows: int, dtype: torch.dtype) -> int:
    """The address of a parameter that is a tensor of one number a row."""
    if value.dtype is not dtype or value.shape != (rows,) or not value.is_contiguous():
        raise ValueError(f"{name} must be a number or a contiguous {dtype} tensor [rows]")
    return value.data_ptr()


def sample_tokens(logits: torch.Tensor, u: torch.Tensor, temperature: "float | torch.Tensor" = 1.0,
                  top_k: "int | torch.Tensor" = 0, top_p: "float | torch.Tensor" = 1.0,
                  min_p: "float | torch.Tensor" = 0.0, out: tuple | None = None, stream=None):
    """Draw a token for each row of logits from given uniform numbers
    (tpa_sample_tokens): temperature, then top-k, top-p and min-p.

    logits [N, V] fp32 or bf16 with unit column stride, V <= 2^24, u [N] fp32 in [0, 1).  Each parameter is a number or a tensor
    [N] (fp32, top_k int32): a temperature of 0 takes the largest logit; top_k <= 0, top_p = 1 and min_p = 0 keep all.
    Returns tokens [N] int32 and their log-probabilities in the distribution that they were drawn from, [N] fp32."""
    f32, i32, T = torch.float32, torch.int32, torch.Tensor
    bf16 = logits.dtype is torch.bfloat16
    if logits.dim() != 2 or not (bf16 or logits.dtype is f32) or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be fp32 or bf16 [rows, vocabulary] with unit column stride")
    N, V = logits.shape
    _int32("the number of rows", N)
    _int32("the vocabulary", V)
    if u.dtype is not f32 or u.shape != (N,) or not u.is_contiguous():
        raise ValueError("u must be a contiguous fp32 tensor [rows]")
    t = p = m = k = None  # the ones that are tensors
    t_at = p_at = m_at = k_at = 0
    if isinstance(temperature, T):
        t, t_at, temperature = temperature, _row_parameter("temperature", temperature, N, f32), 1.0
    if isinstance(top_k, T):
        k, k_at, top_k = top_k, _row_parameter("top_k", top_k, N, i32), 0
    if isinstance(top_p, T):
        p, p_at, top_p = top_p, _row_parameter("top_p", top_p, N, f32), 1.0
    if isinstance(min_p, T):
        m, m_at, min_p = min_p, _row_parameter("min_p", min_p, N, f32), 0.0
    params = SAMPLE_PARAMS.pack(t_at, p_at, m_at, k_at, temperature, top_p, min_p, _int32("top_k", top_k))
    if out is None:
        st = _launch_stream(stream, logits, u, t, p, m, k)
        tokens, logp = _new(stream, (N,), i32, logits.device), _new(stream, (N,), f32, logits.device)
    else:
        tokens, logp = out
        _vector("tokens", tokens, N)
        if logp.dtype is not f32 or logp.shape != (N,) or not logp.is_contiguous():
            raise ValueError("logp must be a contiguous fp32 tensor [rows]")
        st = _launch_stream(stream, logits, u, t, p, m, k, tokens, logp)
    check("tpa_sample_tokens", lib().tpa_sample_tokens(
        logits.data_ptr(), LOGITS_BF16 if bf16 else LOGITS_F32, logits.stride(0) if N > 1 else V, N, V, params, u.data_ptr(),
        tokens.data_ptr(), logp.data_ptr(), st))
    return tokens, logp


def sync_status(stream=None) -> None:
    """Synchronise the stream and raise if any kernel reported a device-side failure."""
    check("tpa_sync_status", lib().tpa_sync_status(_stream_ptr(stream)))


def wait_probe(limit_ns: int, arrive: bool, stream=None) -> None:
    """Launch the bounded-wait diagnostic (tpa_wait_probe): with ``arrive``
    False its one wait runs out after about ``limit_ns`` and the next
    ``sync_status`` raises TPA_ERR_DEVICE_TIMEOUT."""
    check("tpa_wait_probe", lib().tpa_wait_probe(int(limit_ns), 1 if arrive else 0, _stream_ptr(stream)))


def device_check() -> None:
    check("tpa_device_check", lib().tpa_device_check())
