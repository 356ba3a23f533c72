"""ctypes binding of libspecverify.so (argument marshalling only).

Every function here checks tensor devices, dtypes and shapes, then calls the C
ABI declared in include/spec_verify.h with raw device pointers and the current
CUDA stream.  All computation happens in the library's CUDA kernels; there is
no CPU or PyTorch fallback.  Importing this module raises if the library has
not been built (see ``speculative_decoding_verify_07_gb300.build``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libspecverify.so")

SPEC_F32 = 0
SPEC_BF16 = 1
SPEC_E4M3 = 2

SPEC_OK = 0
SPEC_E_NULL = -1
SPEC_E_DIM = -2
SPEC_E_DTYPE = -3
SPEC_E_ALIGN = -4
SPEC_E_WORKSPACE = -5
SPEC_E_CUDA = -6
SPEC_E_ARCH = -7

F_MARGIN_ACCEPT = 1
F_MARGIN_DRAW = 2
F_MARGIN_TOPP = 4
F_NAN = 8
F_BAD_TOKEN = 16
F_BAD_PARAM = 32
F_RESIDUAL_EMPTY = 64
F_BAD_IDX = 128
F_TIMEOUT = 256

SPEC_MAX_V = 524288
SPEC_MAX_K = 16
SPEC_MAX_CONV = 8


# spec_cache_t of include/spec_forward.h, as bytes: k_pages, v_pages, k_exp, v_exp, page_table, cu_tokens, kv_len;
# page_stride, exp_stride; dtype, B, max_pages, pages, heads, page_size, head_dim.
CACHE_T = struct.Struct("@7Q2q7i")
# spec_conv_t of include/spec_hybrid.h: x, weight, bias, state, slot, lens, y, states, last, last_slot, flags; x_row,
# x_tok; dtype, B, T, C, width, slots, last_slots, silu.
CONV_T = struct.Struct("@11Q2q8i")
# spec_scan_t of include/spec_hybrid.h: x, dt, z, b, c, a, skip, dt_bias, state, slot, lens, y, states, last, last_slot,
# flags; row and token strides of x, dt, z, then row, token and group strides of b, c; dtype, B, T, D, N, groups, slots,
# last_slots, softplus.
SCAN_T = struct.Struct("@16Q12q9i4x")


class SpecError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


def _load(path=_LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing; build it with "
            "`python -m speculative_decoding_verify_07_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
    lib.spec_verify_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_verify_workspace_size.restype = sz
    u32 = ctypes.c_uint32
    lib.spec_verify.argtypes = [vp, i32, vp, vp, vp, u64, u32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.spec_verify.restype = i32
    lib.spec_commit.argtypes = [vp, vp, vp, vp, vp, vp] + [i32] * 9 + [vp, vp]
    lib.spec_commit.restype = i32
    lib.spec_commit_swap.argtypes = [vp, vp, vp, vp, vp, vp, vp] + [i32] * 9 + [vp, vp]
    lib.spec_commit_swap.restype = i32
    lib.spec_verify_commit.argtypes = ([vp, i32, vp, vp, vp, u64, u32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz]
                                       + [vp] * 5 + [i32] * 7 + [vp])
    lib.spec_verify_commit.restype = i32
    lib.spec_verify_noalloc.argtypes = [vp, i32, vp, vp, vp, u64, u32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.spec_verify_noalloc.restype = i32
    lib.spec_draft_workspace_size.argtypes = [i32, i32]
    lib.spec_draft_workspace_size.restype = sz
    lib.spec_draft_sample.argtypes = [vp, i32, vp, u64, u32, u32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.spec_draft_sample.restype = i32
    i64, cache = ctypes.c_int64, ctypes.c_char_p
    lib.spec_cache_write.argtypes = [vp, vp, i32, i64, i32, cache, vp, vp]
    lib.spec_cache_write.restype = i32
    lib.spec_cache_read.argtypes = [vp, vp, i32, cache, vp, vp]
    lib.spec_cache_read.restype = i32
    lib.spec_attend_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_attend_workspace_size.restype = sz
    lib.spec_attend.argtypes = [vp, i64, i32, i32, ctypes.c_float, i32, cache, vp, vp, vp, vp, sz, vp]
    lib.spec_attend.restype = i32
    lib.spec_recur_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_recur_workspace_size.restype = sz
    lib.spec_recur.argtypes = [vp, i64, i64, vp, i64, i64, i32, vp, vp, i32, vp, i32, i32, i32, vp, i32, vp, vp, i32,
                               vp, vp, sz, vp]
    lib.spec_recur.restype = i32
    lib.spec_recur_backward.argtypes = [vp, i64, i64, vp, i32, vp, vp, i32, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp,
                                        vp, vp, sz, vp]
    lib.spec_recur_backward.restype = i32
    lib.spec_conv.argtypes = [ctypes.c_char_p, vp]
    lib.spec_conv.restype = i32
    lib.spec_scan_workspace_size.argtypes = [i32] * 4
    lib.spec_scan_workspace_size.restype = sz
    lib.spec_scan.argtypes = [ctypes.c_char_p, vp, sz, vp]
    lib.spec_scan.restype = i32
    lib.spec_attend_shared_workspace_size.argtypes = [i32] * 5
    lib.spec_attend_shared_workspace_size.restype = sz
    lib.spec_attend_shared.argtypes = [vp, i64, i32, i32, ctypes.c_float, i32, cache, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.spec_attend_shared.restype = i32
    lib.spec_philox4x32_10.argtypes = [vp, u64, vp, ctypes.c_int64, vp]
    lib.spec_philox4x32_10.restype = i32
    lib.spec_status_string.argtypes = [i32]
    lib.spec_status_string.restype = ctypes.c_char_p
    lib.spec_version.argtypes = []
    lib.spec_version.restype = i32
    return lib


LIB = _load()
LIB_PATH = _LIB_PATH


def status_string(code: int) -> str:
    return LIB.spec_status_string(int(code)).decode()


def version() -> int:
    return int(LIB.spec_version())


def workspace_size(B: int, k: int, V: int) -> int:
    return int(LIB.spec_verify_workspace_size(int(B), int(k), int(V)))


def row_block(total_rows: int, world: int, rank: int):
    """Rows [lo, hi) of a batch of `total_rows` that rank `rank` of `world`
    verifies, as contiguous blocks (the first total_rows % world ranks take
    one row more).  The rank passes row_base = lo, so that every row draws the
    random numbers of its place in the whole batch and the shards together
    give exactly the single-call result."""
    if world < 1 or not 0 <= rank < world or total_rows < 0:
        raise ValueError(f"bad shard: {total_rows} rows, rank {rank} of {world}")
    base, extra = divmod(int(total_rows), int(world))
    lo = rank * base + min(rank, extra)
    return lo, lo + base + (1 if rank < extra else 0)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def make_params(temperature, top_k, top_p, device) -> torch.Tensor:
    """Pack per-row (temperature, top_k, top_p) into the [B, 4] int32 layout of spec_params_t."""
    T = torch.as_tensor(temperature, dtype=torch.float32).reshape(-1)
    K = torch.as_tensor(top_k, dtype=torch.int32).reshape(-1)
    P = torch.as_tensor(top_p, dtype=torch.float32).reshape(-1)
    z = torch.zeros_like(K)
    packed = torch.stack([T.view(torch.int32), K, P.view(torch.int32), z], dim=1).contiguous()
    return packed.to(device)


class VerifyOutputs:
    def __init__(self, B: int, k: int, device):
        self.tokens = torch.empty((B, k + 1), dtype=torch.int32, device=device)
        self.accept_len = torch.empty((B,), dtype=torch.int32, device=device)
        self.logprobs = torch.empty((B, k + 1), dtype=torch.float32, device=device)
        self.alpha = torch.empty((B, max(k, 0)), dtype=torch.float32, device=device)
        self.flags = torch.empty((B,), dtype=torch.int32, device=device)   # uint32 bit pattern


def new_workspace(B: int, k: int, V: int, device) -> torch.Tensor:
    """A zero-filled workspace (the library leaves it zero-filled after each call)."""
    n = workspace_size(B, k, V)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def spec_verify(logits: torch.Tensor, draft_probs, draft_tokens, params: torch.Tensor, seed: int,
                out: VerifyOutputs | None = None, workspace: torch.Tensor | None = None,
                stream=None, row_base: int = 0) -> VerifyOutputs:
    """Run the verify step; inputs and outputs are CUDA tensors (see spec_verify.h).

    logits [B, k+1, V] float32 or bfloat16; draft_probs [B, k, V] float32;
    draft_tokens [B, k] int32; params [B, 4] int32 from make_params().
    row_base: the stream row of this batch's first row (row r draws as row
    row_base + r), so that a batch split into row blocks reproduces the
    whole batch's draws.
    """
    if logits.dim() != 3:
        raise ValueError("logits must be [B, k+1, V]")
    B, k1, V = logits.shape
    k = k1 - 1
    dev = logits.device
    if logits.dtype == torch.float32:
        dt = SPEC_F32
    elif logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    else:
        raise TypeError("logits must be float32 or bfloat16")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    if k > 0:
        _check(draft_probs, "draft_probs", torch.float32, (B, k, V), dev)
        _check(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _check(params, "params", torch.int32, (B, 4), dev)
    if out is None:
        out = VerifyOutputs(B, k, dev)
    if workspace is None:
        workspace = new_workspace(B, k, V, dev)
    rc = LIB.spec_verify(_ptr(logits), dt, _ptr(draft_probs) if k > 0 else None,
                         _ptr(draft_tokens) if k > 0 else None, _ptr(params),
                         ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                         ctypes.c_uint32(int(row_base) & 0xFFFFFFFF), B, k, V,
                         _ptr(out.tokens), _ptr(out.accept_len), _ptr(out.logprobs),
                         _ptr(out.alpha) if k > 0 else None, _ptr(out.flags),
                         _ptr(workspace), workspace.numel(), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_verify")
    return out


def spec_verify_noalloc(logits: torch.Tensor, draft_probs, draft_tokens, params: torch.Tensor,
                        seed: int, out: VerifyOutputs | None = None, stream=None,
                        row_base: int = 0) -> VerifyOutputs:
    """spec_verify with the library's own scratch array instead of a workspace.

    For callers that cannot allocate device scratch; the library allocates
    nothing either (see spec_verify_noalloc in spec_verify.h for the size
    limit and for why overlapping calls race).  `out` may be preallocated.
    """
    if logits.dim() != 3:
        raise ValueError("logits must be [B, k+1, V]")
    B, k1, V = logits.shape
    k = k1 - 1
    dev = logits.device
    if logits.dtype == torch.float32:
        dt = SPEC_F32
    elif logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    else:
        raise TypeError("logits must be float32 or bfloat16")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    if k > 0:
        _check(draft_probs, "draft_probs", torch.float32, (B, k, V), dev)
        _check(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _check(params, "params", torch.int32, (B, 4), dev)
    if out is None:
        out = VerifyOutputs(B, k, dev)
    rc = LIB.spec_verify_noalloc(_ptr(logits), dt, _ptr(draft_probs) if k > 0 else None,
                                 _ptr(draft_tokens) if k > 0 else None, _ptr(params),
                                 ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                                 ctypes.c_uint32(int(row_base) & 0xFFFFFFFF), B, k, V,
                                 _ptr(out.tokens), _ptr(out.accept_len), _ptr(out.logprobs),
                                 _ptr(out.alpha) if k > 0 else None, _ptr(out.flags), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_verify_noalloc")
    return out


def _commit_dims(verify_rec, verify_conv, cache_rec, cache_conv):
    """(L, B, S, H, Dk, Dv, W, C, slots) of the commit buffers, checked."""
    if verify_rec is not None:
        L, B, S, H, Dk, Dv = verify_rec.shape
        slots = cache_rec.shape[1]
        if verify_rec.dtype != torch.float32 or cache_rec.dtype != torch.float32:
            raise TypeError("recurrent state must be float32")
        if tuple(cache_rec.shape) != (L, slots, H, Dk, Dv):
            raise ValueError("cache_rec shape mismatch")
    else:
        H = Dk = Dv = 1
    if verify_conv is not None:
        Lc, Bc, Sc, W, C = verify_conv.shape
        if verify_rec is None:
            L, B, S = Lc, Bc, Sc
            slots = cache_conv.shape[1]
        elif (Lc, Bc, Sc) != (L, B, S):
            raise ValueError("verify_conv and verify_rec disagree on [L, B, S]")
        if verify_conv.element_size() != 2 or cache_conv.element_size() != 2:
            raise TypeError("conv state must be a 16-bit type")
        if tuple(cache_conv.shape) != (L, slots, W, C):
            raise ValueError("cache_conv shape mismatch")
    else:
        W = C = 1
    if verify_rec is None and verify_conv is None:
        raise ValueError("nothing to commit")
    for t, nm in ((verify_rec, "verify_rec"), (verify_conv, "verify_conv"), (cache_rec, "cache_rec"),
                  (cache_conv, "cache_conv")):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    return L, B, S, H, Dk, Dv, W, C, slots


def spec_commit(verify_rec, verify_conv, accept_len, cache_slot, cache_rec, cache_conv,
                flags=None, stream=None):
    """Commit accepted states (see spec_commit in spec_verify.h).

    verify_rec [L, B, S, H, Dk, Dv] float32 or None; verify_conv [L, B, S, W, C]
    16-bit (bfloat16/int16) or None; accept_len [B] int32; cache_slot [B] int32
    or None; cache_rec [L, slots, H, Dk, Dv]; cache_conv [L, slots, W, C].
    """
    L, B, S, H, Dk, Dv, W, C, slots = _commit_dims(verify_rec, verify_conv, cache_rec, cache_conv)
    dev = accept_len.device
    _check(accept_len, "accept_len", torch.int32, (B,), dev)
    if cache_slot is not None:
        _check(cache_slot, "cache_slot", torch.int32, (B,), dev)
    rc = LIB.spec_commit(_ptr(verify_rec), _ptr(verify_conv), _ptr(accept_len), _ptr(cache_slot),
                         _ptr(cache_rec), _ptr(cache_conv), L, B, S, H, Dk, Dv, W, C, slots,
                         _ptr(flags), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_commit")


def spec_verify_commit(logits: torch.Tensor, draft_probs, draft_tokens, params: torch.Tensor, seed: int,
                       verify_rec, verify_conv, cache_slot, cache_rec, cache_conv,
                       out: VerifyOutputs | None = None, workspace: torch.Tensor | None = None,
                       stream=None, row_base: int = 0) -> VerifyOutputs:
    """spec_verify and spec_commit in one launch (see spec_verify_commit in
    spec_verify.h): the verify outputs, and each row's accepted state
    copied into its cache slot; S = k + 1 states per row."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, k+1, V]")
    B, k1, V = logits.shape
    k = k1 - 1
    dev = logits.device
    if logits.dtype == torch.float32:
        dt = SPEC_F32
    elif logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    else:
        raise TypeError("logits must be float32 or bfloat16")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    if k > 0:
        _check(draft_probs, "draft_probs", torch.float32, (B, k, V), dev)
        _check(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _check(params, "params", torch.int32, (B, 4), dev)
    L, Bc, S, H, Dk, Dv, W, C, slots = _commit_dims(verify_rec, verify_conv, cache_rec, cache_conv)
    if (Bc, S) != (B, k1):
        raise ValueError("state buffers must be [L, B, k+1, ...]")
    if cache_slot is not None:
        _check(cache_slot, "cache_slot", torch.int32, (B,), dev)
    if out is None:
        out = VerifyOutputs(B, k, dev)
    if workspace is None:
        workspace = new_workspace(B, k, V, dev)
    rc = LIB.spec_verify_commit(_ptr(logits), dt, _ptr(draft_probs) if k > 0 else None,
                                _ptr(draft_tokens) if k > 0 else None, _ptr(params),
                                ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                                ctypes.c_uint32(int(row_base) & 0xFFFFFFFF), B, k, V,
                                _ptr(out.tokens), _ptr(out.accept_len), _ptr(out.logprobs),
                                _ptr(out.alpha) if k > 0 else None, _ptr(out.flags),
                                _ptr(workspace), workspace.numel(),
                                _ptr(verify_rec), _ptr(verify_conv), _ptr(cache_slot), _ptr(cache_rec),
                                _ptr(cache_conv), L, H, Dk, Dv, W, C, slots, _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_verify_commit")
    return out


def spec_commit_swap(verify_rec, verify_conv, accept_len, slot_of_row, scratch_slot, cache_rec, cache_conv,
                     flags=None, stream=None):
    """Zero-copy commit (see spec_commit_swap in spec_verify.h).

    verify_rec [L, B, S-1, H, Dk, Dv] float32 or None; verify_conv [L, B, S-1, W, C]
    16-bit or None: the first S - 1 states of each row; the last state of row
    r is already in cache slot scratch_slot[r].  slot_of_row and scratch_slot
    [B] int32 are updated in place (a fully accepted row trades them).
    """
    ref = verify_rec if verify_rec is not None else verify_conv
    if ref is None:
        raise ValueError("nothing to commit")
    L, B, Sm1 = ref.shape[:3]
    S = Sm1 + 1
    if verify_rec is not None:
        _, _, _, H, Dk, Dv = verify_rec.shape
        slots = cache_rec.shape[1]
        if verify_rec.dtype != torch.float32 or cache_rec.dtype != torch.float32:
            raise TypeError("recurrent state must be float32")
        if tuple(cache_rec.shape) != (L, slots, H, Dk, Dv):
            raise ValueError("cache_rec shape mismatch")
    else:
        H = Dk = Dv = 1
    if verify_conv is not None:
        _, _, _, W, C = verify_conv.shape
        if verify_rec is None:
            slots = cache_conv.shape[1]
        if tuple(verify_conv.shape[:3]) != (L, B, Sm1):
            raise ValueError("verify_conv and verify_rec disagree on [L, B, S-1]")
        if verify_conv.element_size() != 2 or cache_conv.element_size() != 2:
            raise TypeError("conv state must be a 16-bit type")
        if tuple(cache_conv.shape) != (L, slots, W, C):
            raise ValueError("cache_conv shape mismatch")
    else:
        W = C = 1
    for t, nm in ((verify_rec, "verify_rec"), (verify_conv, "verify_conv"), (cache_rec, "cache_rec"),
                  (cache_conv, "cache_conv")):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    dev = accept_len.device
    _check(accept_len, "accept_len", torch.int32, (B,), dev)
    _check(slot_of_row, "slot_of_row", torch.int32, (B,), dev)
    _check(scratch_slot, "scratch_slot", torch.int32, (B,), dev)
    rc = LIB.spec_commit_swap(_ptr(verify_rec), _ptr(verify_conv), _ptr(accept_len), _ptr(slot_of_row),
                              _ptr(scratch_slot), _ptr(cache_rec), _ptr(cache_conv), L, B, S, H, Dk, Dv, W, C,
                              slots, _ptr(flags), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_commit_swap")


class DraftOutputs:
    def __init__(self, B: int, V: int, device, with_q: bool = True):
        self.q = torch.empty((B, V), dtype=torch.float32, device=device) if with_q else None
        self.tokens = torch.empty((B,), dtype=torch.int32, device=device)
        self.logprobs = torch.empty((B,), dtype=torch.float32, device=device)
        self.flags = torch.empty((B,), dtype=torch.int32, device=device)   # uint32 bit pattern


def draft_workspace_size(B: int, V: int) -> int:
    return int(LIB.spec_draft_workspace_size(int(B), int(V)))


def new_draft_workspace(B: int, V: int, device) -> torch.Tensor:
    """A zero-filled workspace for spec_draft_sample."""
    return torch.zeros(max(draft_workspace_size(B, V), 16), dtype=torch.uint8, device=device)


def spec_draft_sample(logits: torch.Tensor, params: torch.Tensor, seed: int, pos: int,
                      out: DraftOutputs | None = None, workspace: torch.Tensor | None = None,
                      stream=None, row_base: int = 0, with_q: bool = True) -> DraftOutputs:
    """One draft step (see spec_draft_sample in spec_verify.h): logits [B, V]
    float32 or bfloat16, params [B, 4] int32 from make_params(); draws x ~ q
    and writes q (unless with_q is False)."""
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    B, V = logits.shape
    dev = logits.device
    if logits.dtype == torch.float32:
        dt = SPEC_F32
    elif logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    else:
        raise TypeError("logits must be float32 or bfloat16")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    _check(params, "params", torch.int32, (B, 4), dev)
    if out is None:
        out = DraftOutputs(B, V, dev, with_q)
    if out.q is not None:
        _check(out.q, "q", torch.float32, (B, V), dev)
    if workspace is None:
        workspace = new_draft_workspace(B, V, dev)
    rc = LIB.spec_draft_sample(_ptr(logits), dt, _ptr(params), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                               ctypes.c_uint32(int(row_base) & 0xFFFFFFFF), ctypes.c_uint32(int(pos) & 0xFFFFFFFF),
                               B, V, _ptr(out.q), _ptr(out.tokens), _ptr(out.logprobs), _ptr(out.flags),
                               _ptr(workspace), workspace.numel(), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_draft_sample")
    return out


def philox4x32_10(ctr: torch.Tensor, seed: int, stream=None) -> torch.Tensor:
    """Device Philox4x32-10 of a [n, 4] int32 (bit pattern) counter tensor."""
    if ctr.dim() != 2 or ctr.shape[1] != 4 or ctr.dtype != torch.int32 or not ctr.is_contiguous():
        raise ValueError("ctr must be a contiguous [n, 4] int32 tensor")
    out = torch.empty_like(ctr)
    rc = LIB.spec_philox4x32_10(_ptr(ctr), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)), _ptr(out),
                                ctr.shape[0], _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_philox4x32_10")
    return out


# The forward's sequence mixers (include/spec_forward.h).  A step makes several of
# these calls a layer, so their checks read each attribute of a tensor once.

_POOL_DTYPES = {torch.bfloat16: SPEC_BF16, torch.float8_e4m3fn: SPEC_E4M3}
_IO_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16}
# The device's current stream without the Stream object around it, where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _io_dtype(t, name):
    dt = _IO_DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return dt


def _expect(t, name, dtype, shape, dev):
    """_check for a call's small tensors; the message is made by _check."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check(t, name, dtype, shape, dev)


def _page_stride(a, b, names, per_page):
    """Elements from page to page of two pools whose pages are dense inside."""
    if a.is_contiguous() and b.is_contiguous():
        return per_page
    strides = []
    for t, name in zip((a, b), names):
        inner = 1
        for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
            if size != 1 and stride != inner:
                raise ValueError(f"{name} must be dense within a page")
            inner *= size
        strides.append(t.stride(0) if t.shape[0] > 1 else per_page)
    if a.shape[0] > 1 and strides[0] != strides[1]:
        raise ValueError(f"{names[0]} and {names[1]} must have the same page stride")
    if strides[0] < per_page:
        raise ValueError(f"{names[0]} has overlapping pages")
    return strides[0]


def _cache_view(cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp, v_exp, flags):
    """(spec_cache_t, B, heads, head_dim) of a batch's tensors, checked.  The
    bytes hold raw pointers: the tensors outlive the call that they are made for."""
    dt = _POOL_DTYPES.get(k_pages.dtype)
    if dt is None:
        raise TypeError("the cache must be bfloat16 or float8_e4m3fn")
    shape, dev = k_pages.shape, k_pages.device
    if len(shape) != 4:
        raise ValueError("k_pages must be [pages, heads, page_size, head_dim]")
    pages, heads, page_size, dim = shape
    if v_pages.shape != shape or v_pages.dtype != k_pages.dtype or v_pages.device != dev:
        raise ValueError("v_pages must be like k_pages")
    if cu_tokens.dim() != 1 or page_table.dim() != 2:
        raise ValueError("cu_tokens must be [B + 1] and page_table [B, max_pages]")
    B, max_pages = page_table.shape
    i32 = torch.int32
    _expect(cu_tokens, "cu_tokens", i32, (B + 1,), dev)
    _expect(kv_len, "kv_len", i32, (B,), dev)
    _expect(page_table, "page_table", i32, (B, max_pages), dev)
    if flags is not None:
        _expect(flags, "flags", i32, (B,), dev)
    ke = ve = exp_stride = 0
    if dt == SPEC_E4M3:
        for t, name in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            if t is None:
                raise ValueError(f"an e4m3 cache needs {name}")
            if t.dtype is not torch.uint8 or t.device != dev or t.shape != (pages, heads, page_size):
                raise ValueError(f"{name} must be uint8 [pages, heads, page_size] on {dev}")
        exp_stride = _page_stride(k_exp, v_exp, ("k_exp", "v_exp"), heads * page_size)
        ke, ve = k_exp.data_ptr(), v_exp.data_ptr()
    elif k_exp is not None or v_exp is not None:
        raise ValueError("a bfloat16 cache has no exponents")
    page_stride = _page_stride(k_pages, v_pages, ("k_pages", "v_pages"), heads * page_size * dim)
    view = CACHE_T.pack(k_pages.data_ptr(), v_pages.data_ptr(), ke, ve, page_table.data_ptr(), cu_tokens.data_ptr(),
                        kv_len.data_ptr(), page_stride, exp_stride, dt, B, max_pages, pages, heads, page_size, dim)
    return view, B, heads, dim


def _token_stride(t, name):
    """Elements from token to token of [N, heads, dim] with dense tokens."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [N, heads, head_dim]")
    n, h, d = t.shape
    token, head, one = t.stride()
    if (d > 1 and one != 1) or (h > 1 and head != d):
        raise ValueError(f"{name} must be dense within a token")
    if n > 1 and token < h * d:
        raise ValueError(f"{name} has overlapping tokens")
    return token if n > 1 else h * d


def _at(t):
    return None if t is None else t.data_ptr()


def _queue(stream, dev):
    """The raw stream that a call goes to: the given one, or the device's current
    one.  Kernels read what they are given, so tensors elsewhere are refused."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not on {dev}")
    return _raw_stream(dev.index) if stream is None else stream.cuda_stream


def _space(workspace, dev):
    """(address, bytes) of a given workspace."""
    if workspace.dtype is not torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous uint8 on {dev}")
    return workspace.data_ptr(), workspace.numel()


def _empty(shape, dtype, dev, stream):
    """What a call allocates for itself is allocated on the stream that it runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _on(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _done(rc, what):
    if rc != SPEC_OK:
        raise SpecError(rc, what)


def spec_cache_write(k, v, cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp=None, v_exp=None, flags=None,
                     stream=None):
    """Put new tokens' keys and values into the paged cache (see spec_cache_write
    in spec_forward.h).

    k, v [N, heads, head_dim] float32 or bfloat16 (tokens may be strided);
    cu_tokens [B + 1], kv_len [B], page_table [B, max_pages] int32; k_pages,
    v_pages [pages, heads, page_size, head_dim] bfloat16 or float8_e4m3fn, the
    latter with k_exp, v_exp [pages, heads, page_size] uint8; flags [B] int32.
    """
    view, _, heads, dim = _cache_view(cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp, v_exp, flags)
    dt, stride, shape, dev = _io_dtype(k, "k"), _token_stride(k, "k"), k.shape, k.device
    if shape[1] != heads or shape[2] != dim or dev != k_pages.device:
        raise ValueError(f"k must be [N, {heads}, {dim}] on {k_pages.device}")
    if v.shape != shape or v.dtype != k.dtype or v.device != dev or (v.stride() != k.stride() and _token_stride(v, "v") != stride):
        raise ValueError("v must be like k")
    rc = LIB.spec_cache_write(k.data_ptr(), v.data_ptr(), dt, stride, shape[0], view, _at(flags), _queue(stream, dev))
    _done(rc, "spec_cache_write")


def spec_cache_read(tokens, cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp=None, v_exp=None, k=None, v=None,
                    flags=None, stream=None):
    """Read `tokens` = cu_tokens[B] packed tokens back as bfloat16 (see
    spec_cache_read in spec_forward.h); returns (k, v), each [tokens, heads,
    head_dim]."""
    view, _, heads, dim = _cache_view(cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp, v_exp, flags)
    shape, dev = (int(tokens), heads, dim), k_pages.device
    if k is None:
        k = _empty(shape, torch.bfloat16, dev, stream)
    else:
        _expect(k, "k", torch.bfloat16, shape, dev)
    if v is None:
        v = _empty(shape, torch.bfloat16, dev, stream)
    else:
        _expect(v, "v", torch.bfloat16, shape, dev)
    rc = LIB.spec_cache_read(k.data_ptr(), v.data_ptr(), shape[0], view, _at(flags), _queue(stream, dev))
    _done(rc, "spec_cache_read")
    return k, v


def new_attend_workspace(heads: int, group: int, head_dim: int, device) -> torch.Tensor:
    """A zero-filled workspace for spec_attend: any batch of a cache of `heads`
    heads of head_dim, each read by `group` query heads; one stream."""
    n = int(LIB.spec_attend_workspace_size(int(heads), int(group), int(head_dim)))
    if n == 0:
        raise ValueError(f"spec_attend takes no {heads} heads of {head_dim} read by {group}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _attend_io(q, out, lse, heads, head_dim, dev, stream):
    """(token stride of q, N, query heads, out, lse) of an attention's arrays, checked."""
    stride = _token_stride(q, "q")
    N, hq, dim = q.shape
    if q.dtype is not torch.bfloat16:
        raise TypeError("q must be bfloat16")
    if dim != head_dim or hq % heads or q.device != dev:
        raise ValueError(f"q must be [N, a multiple of {heads}, {head_dim}] on {dev}")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    else:
        _expect(out, "out", torch.bfloat16, (N, hq, dim), dev)
    if lse is None:
        lse = _empty((N, hq), torch.float32, dev, stream)
    else:
        _expect(lse, "lse", torch.float32, (N, hq), dev)
    return stride, N, hq, out, lse


def spec_attend(q, cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp=None, v_exp=None, *, max_tokens, scale=None,
                out=None, lse=None, flags=None, workspace=None, stream=None):
    """Causal attention of each row's new tokens over its paged cache (see
    spec_attend in spec_forward.h); the cache as for spec_cache_write, which
    has put the new tokens in.

    q [N, heads * group, head_dim] bfloat16 (tokens may be strided); scale
    defaults to head_dim ** -0.5; max_tokens is the largest number of new
    tokens of a row.  Without a workspace the call makes one and zeroes it (40 MB
    for heads of 128): a loop keeps one.  Returns (out [N, heads * group, head_dim] bfloat16,
    lse [N, heads * group] float32).
    """
    view, _, heads, head_dim = _cache_view(cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp, v_exp, flags)
    dev, dim = k_pages.device, head_dim
    stride, N, hq, out, lse = _attend_io(q, out, lse, heads, head_dim, dev, stream)
    if workspace is None:
        with _on(stream):
            workspace = new_attend_workspace(heads, hq // heads, dim, dev)
    rc = LIB.spec_attend(q.data_ptr(), stride, N, hq // heads, dim ** -0.5 if scale is None else scale, max_tokens, view,
                         out.data_ptr(), lse.data_ptr(), _at(flags), *_space(workspace, dev), _queue(stream, dev))
    _done(rc, "spec_attend")
    return out, lse


def recur_workspace_size(B: int, T: int, D: int) -> int:
    return int(LIB.spec_recur_workspace_size(int(B), int(T), int(D)))


def new_recur_workspace(B: int, T: int, D: int, device) -> torch.Tensor:
    """A zero-filled workspace for spec_recur and spec_recur_backward."""
    return torch.zeros(max(recur_workspace_size(B, T, D), 256), dtype=torch.uint8, device=device)


def _recur_strides(t, name, shape, dtype, dev):
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {dev}")
    row, tok, one = t.stride()
    if shape[2] > 1 and one != 1:
        raise ValueError(f"{name} must have dense channels")
    return row, tok


def _recur_rows(state, slot, lens, flags, B, D, dev):
    """The per-row arguments, checked; the number of states."""
    slots = 0
    if state is not None:
        if state.dim() != 2:
            raise ValueError("state must be [slots, D]")
        slots = state.shape[0]
        _expect(state, "state", torch.float32, (slots, D), dev)
    for t, name in ((slot, "slot"), (lens, "lens"), (flags, "flags")):
        if t is not None:
            _expect(t, name, torch.int32, (B,), dev)
    return slots


def spec_recur(g, x, state=None, slot=None, lens=None, *, h=None, h_dtype=torch.float32, last=None, last_slot=None,
               flags=None, workspace=None, stream=None):
    """h_t = exp(g_t) h_{t-1} + x_t (see spec_recur in spec_forward.h).

    g, x [B, T, D] float32 or bfloat16 (rows and tokens may be strided); state
    [slots, D] float32, slot [B], lens [B] int32, each or None.  Returns (h
    [B, T, D] of h_dtype, last).  last [B, D] float32 is made where None is
    given; last=state, last_slot=slot updates a cache in place.
    """
    if g.dim() != 3:
        raise ValueError("g must be [B, T, D]")
    shape, dev, dt = g.shape, g.device, _io_dtype(g, "g")
    B, T, D = shape
    g_row, g_tok = _recur_strides(g, "g", shape, g.dtype, dev)
    x_row, x_tok = _recur_strides(x, "x", shape, g.dtype, dev)
    slots = _recur_rows(state, slot, lens, flags, B, D, dev)
    if h is None:
        h = _empty(shape, h_dtype, dev, stream)
    else:
        _expect(h, "h", h.dtype, shape, dev)
    if last is None:
        last = _empty((B, D), torch.float32, dev, stream)
        last_slots = B
    else:
        last_slots = last.shape[0]
        _expect(last, "last", torch.float32, (last_slots, D), dev)
    if last_slot is not None:
        _expect(last_slot, "last_slot", torch.int32, (B,), dev)
    if workspace is None:
        with _on(stream):
            workspace = new_recur_workspace(B, T, D, dev)
    rc = LIB.spec_recur(g.data_ptr(), g_row, g_tok, x.data_ptr(), x_row, x_tok, dt, _at(state), _at(slot), slots, _at(lens),
                        B, T, D, h.data_ptr(), _io_dtype(h, "h"), last.data_ptr(), _at(last_slot), last_slots, _at(flags),
                        *_space(workspace, dev), _queue(stream, dev))
    _done(rc, "spec_recur")
    return h, last


def spec_recur_backward(g, h, dh, state=None, slot=None, lens=None, d_last=None, *, dg=None, dx=None, d_state=None,
                        flags=None, workspace=None, stream=None):
    """The gradients of spec_recur (see spec_recur_backward in spec_forward.h):
    g, state, slot, lens as given to it, h as it wrote it, dh [B, T, D] of g's
    dtype, d_last [B, D] float32 or None.  Returns (dg, dx, d_state)."""
    if g.dim() != 3:
        raise ValueError("g must be [B, T, D]")
    shape, dev, dt = g.shape, g.device, _io_dtype(g, "g")
    B, T, D = shape
    g_row, g_tok = _recur_strides(g, "g", shape, g.dtype, dev)
    _expect(dh, "dh", g.dtype, shape, dev)
    _expect(h, "h", h.dtype, shape, dev)
    slots = _recur_rows(state, slot, lens, flags, B, D, dev)
    if d_last is not None:
        _expect(d_last, "d_last", torch.float32, (B, D), dev)
    if dg is None:
        dg = _empty(shape, g.dtype, dev, stream)
    else:
        _expect(dg, "dg", g.dtype, shape, dev)
    if dx is None:
        dx = _empty(shape, g.dtype, dev, stream)
    else:
        _expect(dx, "dx", g.dtype, shape, dev)
    if d_state is None:
        d_state = _empty((B, D), torch.float32, dev, stream)
    else:
        _expect(d_state, "d_state", torch.float32, (B, D), dev)
    if workspace is None:
        with _on(stream):
            workspace = new_recur_workspace(B, T, D, dev)
    rc = LIB.spec_recur_backward(g.data_ptr(), g_row, g_tok, h.data_ptr(), _io_dtype(h, "h"), dh.data_ptr(), _at(d_last), dt,
                                 _at(state), _at(slot), slots, _at(lens), B, T, D, dg.data_ptr(), dx.data_ptr(),
                                 d_state.data_ptr(), _at(flags), *_space(workspace, dev), _queue(stream, dev))
    _done(rc, "spec_recur_backward")
    return dg, dx, d_state


# The mixers of hybrid targets and of groups of samples (include/spec_hybrid.h).

def _address(t):
    return 0 if t is None else t.data_ptr()


def _mixer_out(given, name, shape, dtype, dev, stream):
    if given is None:
        return _empty(shape, dtype, dev, stream)
    _expect(given, name, dtype, shape, dev)
    return given


def _mixer_states(state, states, last, inner, dtype, B, T, dev, stream):
    """state, states and last of a call, checked: (slots, last, last_slots)."""
    slots = 0
    if state is not None:
        slots = state.shape[0]
        _expect(state, "state", dtype, (slots, *inner), dev)
    if states is not None:
        _expect(states, "states", dtype, (B, T, *inner), dev)
    if last is None:
        return slots, _empty((B, *inner), dtype, dev, stream), B
    _expect(last, "last", dtype, (last.shape[0], *inner), dev)
    return slots, last, last.shape[0]


def _mixer_rows(B, dev, **given):
    for name, t in given.items():
        if t is not None:
            _expect(t, name, torch.int32, (B,), dev)


def spec_conv(x, weight, bias=None, state=None, slot=None, lens=None, *, silu=True, y=None, states=None, last=None,
              last_slot=None, flags=None, stream=None):
    """The short causal convolution of a state space layer (see spec_conv in spec_hybrid.h).

    x [B, T, C] float32 or bfloat16 (rows and tokens may be strided); weight [width, C], bias [C] float32; state
    [slots, width - 1, C] of x's dtype, slot [B], lens [B] int32, each or None.  states [B, T, width - 1, C], where given,
    receives the state behind each token.  Returns (y [B, T, C], last).  last [B, width - 1, C] is made where None is
    given; last=state, last_slot=slot updates a cache in place.
    """
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, C] and weight [width, C]")
    shape, dev, dt = x.shape, x.device, _io_dtype(x, "x")
    B, T, C = shape
    width = weight.shape[0]
    if not 2 <= width <= SPEC_MAX_CONV:
        raise ValueError(f"spec_conv takes 2 to {SPEC_MAX_CONV} taps, not {width}")
    x_row, x_tok = _recur_strides(x, "x", shape, x.dtype, dev)
    _expect(weight, "weight", torch.float32, (width, C), dev)
    if bias is not None:
        _expect(bias, "bias", torch.float32, (C,), dev)
    _mixer_rows(B, dev, slot=slot, lens=lens, last_slot=last_slot, flags=flags)
    queue = _queue(stream, dev)
    slots, last, last_slots = _mixer_states(state, states, last, (width - 1, C), x.dtype, B, T, dev, stream)
    y = _mixer_out(y, "y", shape, x.dtype, dev, stream)
    view = CONV_T.pack(x.data_ptr(), weight.data_ptr(), _address(bias), _address(state), _address(slot), _address(lens),
                       y.data_ptr(), _address(states), last.data_ptr(), _address(last_slot), _address(flags), x_row, x_tok, dt,
                       B, T, C, width, slots, last_slots, bool(silu))
    _done(LIB.spec_conv(view, queue), "spec_conv")
    return y, last


def new_scan_workspace(B: int, T: int, D: int, N: int, device) -> torch.Tensor:
    """A workspace for spec_scan: calls of up to B rows of up to T tokens over D channels of N states, one at a time."""
    n = int(LIB.spec_scan_workspace_size(int(B), int(T), int(D), int(N)))
    if n == 0:
        raise ValueError(f"spec_scan takes no {B} rows of {T} tokens over {D} channels of {N} states")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _scan_groups(t, name, shape, dtype, dev):
    """Strides of row, token and group of [B, T, groups, N], N dense."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {dev}")
    *outer, one = t.stride()
    if one != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have dense states")
    return outer


def spec_scan(x, dt, a, b, c, skip=None, z=None, dt_bias=None, state=None, slot=None, lens=None, *, softplus=True, y=None,
              states=None, last=None, last_slot=None, flags=None, workspace=None, stream=None):
    """The selective scan of a state space layer (see spec_scan in spec_hybrid.h).

    x, dt, z [B, T, D] and b, c [B, T, groups, N] float32 or bfloat16 (strided, with dense channels and states); a [D, N],
    skip, dt_bias [D] float32; state [slots, D, N] float32, slot [B], lens [B] int32; z, skip, dt_bias, state, slot, lens
    may be None.  states [B, T, D, N] float32, where given, receives the state behind each token.  Returns (y [B, T, D] of
    x's dtype, last).  last [B, D, N] float32 is made where None is given; last=state, last_slot=slot updates a cache in
    place.
    """
    if x.dim() != 3 or a.dim() != 2 or b.dim() != 4:
        raise ValueError("x must be [B, T, D], a [D, N] and b [B, T, groups, N]")
    shape, dev, kind = x.shape, x.device, _io_dtype(x, "x")
    B, T, D = shape
    N, groups = a.shape[1], b.shape[2]
    strides = [*_recur_strides(x, "x", shape, x.dtype, dev), *_recur_strides(dt, "dt", shape, x.dtype, dev)]
    strides += (0, 0) if z is None else _recur_strides(z, "z", shape, x.dtype, dev)
    for t, name in ((b, "b"), (c, "c")):
        strides += _scan_groups(t, name, (B, T, groups, N), x.dtype, dev)
    f32 = torch.float32
    _expect(a, "a", f32, (D, N), dev)
    for t, name in ((skip, "skip"), (dt_bias, "dt_bias")):
        if t is not None:
            _expect(t, name, f32, (D,), dev)
    _mixer_rows(B, dev, slot=slot, lens=lens, last_slot=last_slot, flags=flags)
    queue = _queue(stream, dev)
    slots, last, last_slots = _mixer_states(state, states, last, (D, N), f32, B, T, dev, stream)
    y = _mixer_out(y, "y", shape, x.dtype, dev, stream)
    if workspace is None:
        with _on(stream):
            workspace = new_scan_workspace(B, T, D, N, dev)
    view = SCAN_T.pack(x.data_ptr(), dt.data_ptr(), _address(z), b.data_ptr(), c.data_ptr(), a.data_ptr(), _address(skip),
                       _address(dt_bias), _address(state), _address(slot), _address(lens), y.data_ptr(), _address(states),
                       last.data_ptr(), _address(last_slot), _address(flags), *strides, kind, B, T, D, N, groups, slots,
                       last_slots, bool(softplus))
    _done(LIB.spec_scan(view, *_space(workspace, dev), queue), "spec_scan")
    return y, last


def new_attend_shared_workspace(tokens: int, rows: int, heads: int, group: int, head_dim: int, device) -> torch.Tensor:
    """A zero-filled workspace for spec_attend_shared: up to `tokens` new tokens in up to `rows` rows over a cache of
    `heads` heads of head_dim, each read by `group` query heads; one stream."""
    n = int(LIB.spec_attend_shared_workspace_size(int(tokens), int(rows), int(heads), int(group), int(head_dim)))
    if n == 0:
        raise ValueError(f"spec_attend_shared takes no {tokens} tokens in {rows} rows over {heads} heads of {head_dim} read by {group}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def spec_attend_shared(q, shared_rows, shared_len, cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp=None, v_exp=None, *,
                       max_tokens, scale=None, out=None, lse=None, flags=None, workspace=None, stream=None):
    """spec_attend for groups of rows that have their first positions in common, which are read once a group (see
    spec_attend_shared in spec_hybrid.h).

    shared_rows [groups + 1] int32: group g are rows shared_rows[g] .. shared_rows[g + 1] - 1; shared_len [groups] int32: the
    positions that they share, read through the page table of the group's first row.  All else as for spec_attend, but
    for the workspace, which new_attend_shared_workspace makes.  It pays for many rows of few tokens behind a long prompt (64
    rows behind 1000 positions, 8 behind 12,000; see the header); otherwise spec_attend is the faster.
    """
    view, B, heads, head_dim = _cache_view(cu_tokens, kv_len, page_table, k_pages, v_pages, k_exp, v_exp, flags)
    dev = k_pages.device
    stride, N, hq, out, lse = _attend_io(q, out, lse, heads, head_dim, dev, stream)
    if shared_len.dim() != 1 or shared_len.shape[0] > B:
        raise ValueError(f"shared_len must be [groups], at most {B} groups")
    groups = shared_len.shape[0]
    _expect(shared_len, "shared_len", torch.int32, (groups,), dev)
    _expect(shared_rows, "shared_rows", torch.int32, (groups + 1,), dev)
    if workspace is None:
        with _on(stream):
            workspace = new_attend_shared_workspace(N, B, heads, hq // heads, head_dim, dev)
    rc = LIB.spec_attend_shared(q.data_ptr(), stride, N, hq // heads, head_dim ** -0.5 if scale is None else scale, max_tokens, view,
                                shared_rows.data_ptr(), shared_len.data_ptr(), groups, out.data_ptr(), lse.data_ptr(), _at(flags),
                                *_space(workspace, dev), _queue(stream, dev))
    _done(rc, "spec_attend_shared")
    return out, lse
