"""Python binding of ``libspecverify.so``: the C ABI in ``include/spec_verify.h``.

Argument marshalling only.  Every step of verification and expansion runs in
the library's HIP kernels; torch supplies device memory and the stream.  There
is no fallback: if the library has not been built (``build.py``) importing the
binding raises.

Same names as the C ABI: ``spec_verify_workspace_bytes``,
``spec_verify_launch``, ``spec_expand_launch``, ``spec_status_string``; plus two convenience wrappers, ``verify`` and
``expand``, that allocate the outputs and call the launchers on torch's current
stream.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspecverify.so")

SPEC_OK, SPEC_EINVAL, SPEC_EDTYPE, SPEC_EALIGN, SPEC_EWORKSPACE, SPEC_ELAUNCH = 0, -1, -2, -3, -4, -5
SPEC_F32, SPEC_BF16 = 0, 1
SPEC_MAX_K = 63
SPEC_MAX_V = 2147418112  # 2^31 - 2^16
SPEC_NOALLOC_SCRATCH_BYTES = 16 << 20
SPEC_MAX_TOP = 32  # most alternatives per row of token_logprobs
SPEC_PHASES_DYNAMIC = 1  # phase_starts value: decisions inside the row pass (dynamic early exit)

EXPORTED = ("spec_verify_workspace_bytes", "spec_verify_plan_phases", "spec_verify_phase_cost",
            "spec_verify_launch", "spec_verify_launch_noalloc",
            "spec_expand_launch", "spec_expand_hidden_launch", "spec_verify_expand_launch",
            "spec_draft_workspace_bytes",
            "spec_draft_sample_launch", "spec_shard_workspace_bytes", "spec_shard_stats_launch",
            "spec_shard_phase_launch", "spec_shard_decide_launch", "spec_shard_draw_launch",
            "spec_logprobs_workspace_bytes", "spec_logprobs_launch", "spec_kv_write_launch",
            "spec_kv_read_launch", "spec_attn_workspace_bytes", "spec_attn_launch",
            "spec_workspace_error", "spec_status_string")


class SpecVerifyArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("target_logits", ctypes.c_void_p), ("t_req_stride", ctypes.c_int64), ("t_row_stride", ctypes.c_int64),
        ("draft_logits", ctypes.c_void_p), ("d_req_stride", ctypes.c_int64), ("d_row_stride", ctypes.c_int64),
        ("draft_tokens", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
        ("seed", ctypes.c_uint64), ("step", ctypes.c_uint32), ("request_base", ctypes.c_uint32),
        ("accepted_counts", ctypes.c_void_p), ("output_tokens", ctypes.c_void_p),
        ("debug_probs", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("phase_event", ctypes.c_void_p), ("phase_starts", ctypes.c_uint64),
        ("draft_row_index", ctypes.c_void_p), ("draft_rows", ctypes.c_int32),
        ("num_drafts", ctypes.c_void_p), ("draft_stats", ctypes.c_void_p),
    ]


class SpecExpandArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("K", ctypes.c_int32), ("H", ctypes.c_int32), ("N_in", ctypes.c_int32),
        ("in_token_ids", ctypes.c_void_p), ("in_positions", ctypes.c_void_p), ("in_start", ctypes.c_void_p),
        ("accepted_counts", ctypes.c_void_p), ("bonus_tokens", ctypes.c_void_p),
        ("verify_output_tokens", ctypes.c_void_p),
        ("mask_token_id", ctypes.c_int32),
        ("target_hidden", ctypes.c_void_p), ("hidden_row_stride", ctypes.c_int64),
        ("mask_hidden", ctypes.c_void_p),
        ("out_token_ids", ctypes.c_void_p), ("out_positions", ctypes.c_void_p),
        ("rejected_mask", ctypes.c_void_p), ("masked_mask", ctypes.c_void_p),
        ("new_token_indices", ctypes.c_void_p), ("hidden_map", ctypes.c_void_p),
        ("out_start", ctypes.c_void_p), ("out_hidden", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("bt_row_stride", ctypes.c_int64),
        ("max_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("slot_mapping", ctypes.c_void_p),
    ]


class SpecDraftArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("N", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
        ("row_index", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
        ("seed", ctypes.c_uint64), ("step", ctypes.c_uint32), ("request_base", ctypes.c_uint32),
        ("tokens", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stats_out", ctypes.c_void_p),
    ]


DRAFT_STATS_BYTES = 16  # one record per (request, position)


class SpecShardArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("G", ctypes.c_int32), ("g", ctypes.c_int32), ("v0", ctypes.c_int32), ("Vs", ctypes.c_int32),
        ("target_logits", ctypes.c_void_p), ("t_req_stride", ctypes.c_int64), ("t_row_stride", ctypes.c_int64),
        ("draft_logits", ctypes.c_void_p), ("d_req_stride", ctypes.c_int64), ("d_row_stride", ctypes.c_int64),
        ("draft_tokens", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
        ("seed", ctypes.c_uint64), ("step", ctypes.c_uint32), ("request_base", ctypes.c_uint32),
        ("records", ctypes.c_void_p), ("masses", ctypes.c_void_p),
        ("accepted_counts", ctypes.c_void_p), ("output_tokens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("num_drafts", ctypes.c_void_p), ("draft_row_index", ctypes.c_void_p), ("draft_rows", ctypes.c_int32),
        ("phase_starts", ctypes.c_uint64), ("phase", ctypes.c_int32),
    ]


class SpecLogprobsArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("R", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("logits", ctypes.c_void_p), ("req_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
        ("tokens", ctypes.c_void_p), ("temperature", ctypes.c_void_p), ("top", ctypes.c_int32),
        ("logprobs", ctypes.c_void_p), ("entropy", ctypes.c_void_p), ("top_ids", ctypes.c_void_p),
        ("top_logprobs", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class SpecKVCache(ctypes.Structure):
    _fields_ = [
        ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("scale_tokens", ctypes.c_int32),
        ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("block_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
        ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("scale_block_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
    ]


class SpecKVWriteArgs(ctypes.Structure):
    _fields_ = [
        ("cache", SpecKVCache), ("N", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("key", ctypes.c_void_p), ("value", ctypes.c_void_p),
        ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
        ("slots", ctypes.c_void_p),
    ]


class SpecKVReadArgs(ctypes.Structure):
    _fields_ = [
        ("cache", SpecKVCache), ("N", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("key", ctypes.c_void_p), ("value", ctypes.c_void_p), ("slots", ctypes.c_void_p),
    ]


class SpecAttnArgs(ctypes.Structure):
    _fields_ = [
        ("cache", SpecKVCache), ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("q_heads", ctypes.c_int32),
        ("max_q", ctypes.c_int32), ("max_ctx", ctypes.c_int32), ("window", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("q_start", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("bt_row_stride", ctypes.c_int64), ("max_blocks", ctypes.c_int32),
        ("sinks", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def _load():
    # torch ships its own HIP runtime under the same SONAME as the system one;
    # loading torch first makes this library bind to that single runtime
    # instead of pulling in a second copy.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libspecverify.so is not built (expected at %s); run rejection_sampling_verify_03_amd/build.py "
            "or __graft_entry__.build()" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    L.spec_verify_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    L.spec_verify_workspace_bytes.restype = ctypes.c_size_t
    L.spec_verify_plan_phases.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_double), ctypes.c_double,
                                          ctypes.c_double]
    L.spec_verify_plan_phases.restype = ctypes.c_uint64
    L.spec_verify_phase_cost.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    L.spec_verify_phase_cost.restype = ctypes.c_double
    L.spec_verify_launch.argtypes = [ctypes.POINTER(SpecVerifyArgs), ctypes.c_void_p]
    L.spec_verify_launch.restype = ctypes.c_int
    L.spec_verify_launch_noalloc.argtypes = [ctypes.POINTER(SpecVerifyArgs), ctypes.c_void_p]
    L.spec_verify_launch_noalloc.restype = ctypes.c_int
    L.spec_workspace_error.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    L.spec_workspace_error.restype = ctypes.c_int
    L.spec_expand_launch.argtypes = [ctypes.POINTER(SpecExpandArgs), ctypes.c_void_p]
    L.spec_expand_launch.restype = ctypes.c_int
    L.spec_verify_expand_launch.argtypes = [ctypes.POINTER(SpecVerifyArgs), ctypes.POINTER(SpecExpandArgs),
                                            ctypes.c_void_p]
    L.spec_verify_expand_launch.restype = ctypes.c_int
    L.spec_expand_hidden_launch.argtypes = [ctypes.POINTER(SpecExpandArgs), ctypes.c_void_p]
    L.spec_expand_hidden_launch.restype = ctypes.c_int
    L.spec_draft_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    L.spec_draft_workspace_bytes.restype = ctypes.c_size_t
    L.spec_draft_sample_launch.argtypes = [ctypes.POINTER(SpecDraftArgs), ctypes.c_void_p]
    L.spec_draft_sample_launch.restype = ctypes.c_int
    L.spec_shard_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    L.spec_shard_workspace_bytes.restype = ctypes.c_size_t
    for name in ("spec_shard_stats_launch", "spec_shard_phase_launch", "spec_shard_decide_launch",
                 "spec_shard_draw_launch"):
        getattr(L, name).argtypes = [ctypes.POINTER(SpecShardArgs), ctypes.c_void_p]
        getattr(L, name).restype = ctypes.c_int
    L.spec_logprobs_workspace_bytes.argtypes = [ctypes.c_int32] * 4
    L.spec_logprobs_workspace_bytes.restype = ctypes.c_size_t
    L.spec_attn_workspace_bytes.argtypes = [ctypes.POINTER(SpecAttnArgs)]
    L.spec_attn_workspace_bytes.restype = ctypes.c_size_t
    for name, struct in (("spec_logprobs_launch", SpecLogprobsArgs), ("spec_kv_write_launch", SpecKVWriteArgs),
                         ("spec_kv_read_launch", SpecKVReadArgs), ("spec_attn_launch", SpecAttnArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(struct), ctypes.c_void_p]
        getattr(L, name).restype = ctypes.c_int
    L.spec_status_string.argtypes = [ctypes.c_int]
    L.spec_status_string.restype = ctypes.c_char_p
    return L


lib = _load()


class SpecError(RuntimeError):
    def __init__(self, status):
        super().__init__(spec_status_string(status))
        self.status = status


# ----------------------------------------------------------------- raw C ABI
def spec_verify_workspace_bytes(B, K, V):
    return int(lib.spec_verify_workspace_bytes(int(B), int(K), int(V)))


def spec_verify_plan_phases(K, survival, sampled_fraction, phase_cost):
    """survival: K+1 floats, survival[k] = probability that a request reaches
    draft position k.  Returns the phase_starts bit mask (0 = one pass)."""
    arr = (ctypes.c_double * (int(K) + 1))(*[float(v) for v in survival])
    return int(lib.spec_verify_plan_phases(int(K), arr, float(sampled_fraction), float(phase_cost)))


def spec_verify_phase_cost(B, K, V, dtype=SPEC_BF16):
    """The price of one early-exit phase boundary for a batch of this shape,
    in row-units (the planner's unit); -1 for an invalid shape."""
    return float(lib.spec_verify_phase_cost(int(B), int(K), int(V), int(dtype)))


def plan_phases(B, K, V, survival, sampled_fraction, dtype=SPEC_BF16):
    """The phase_starts mask the planner picks for this batch shape and
    acceptance curve, with the boundary priced by spec_verify_phase_cost."""
    return spec_verify_plan_phases(K, survival, sampled_fraction, spec_verify_phase_cost(B, K, V, dtype))


def survival_from_accepted(accepted, K):
    """survival[k] = fraction of valid requests whose first k drafts were
    accepted, from a batch of accepted counts (any iterable of ints)."""
    a = [int(v) for v in accepted if int(v) >= 0]
    n = max(len(a), 1)
    return [sum(1 for v in a if v >= k) / n for k in range(int(K) + 1)]


def spec_verify_launch(args, stream_ptr):
    """args: a SpecVerifyArgs; stream_ptr: hipStream_t as an int (0 = null stream)."""
    return int(lib.spec_verify_launch(ctypes.byref(args), stream_ptr))


def spec_verify_launch_noalloc(args, stream_ptr):
    """The same verification with the library's own per-GPU scratch array as
    its workspace (args.workspace ignored); allocates nothing."""
    return int(lib.spec_verify_launch_noalloc(ctypes.byref(args), stream_ptr))


def spec_workspace_error(workspace, stream_ptr=0):
    """Invalid requests of the last verification on this workspace (a device
    tensor or pointer); waits for the stream.  Negative: a spec_status."""
    ptr = workspace.data_ptr() if hasattr(workspace, "data_ptr") else workspace
    return int(lib.spec_workspace_error(ptr, stream_ptr))


def spec_expand_launch(args, stream_ptr):
    return int(lib.spec_expand_launch(ctypes.byref(args), stream_ptr))


def spec_verify_expand_launch(verify_args_, expand_args_, stream_ptr):
    """The verification and the expansion of its outputs as one chained call."""
    return int(lib.spec_verify_expand_launch(ctypes.byref(verify_args_), ctypes.byref(expand_args_), stream_ptr))


def spec_expand_hidden_launch(args, stream_ptr):
    return int(lib.spec_expand_hidden_launch(ctypes.byref(args), stream_ptr))


def spec_draft_workspace_bytes(B, K, V):
    return int(lib.spec_draft_workspace_bytes(int(B), int(K), int(V)))


def spec_draft_sample_launch(args, stream_ptr):
    return int(lib.spec_draft_sample_launch(ctypes.byref(args), stream_ptr))


def spec_shard_workspace_bytes(B, K, Vs):
    return int(lib.spec_shard_workspace_bytes(int(B), int(K), int(Vs)))


def spec_shard_stats_launch(args, stream_ptr):
    return int(lib.spec_shard_stats_launch(ctypes.byref(args), stream_ptr))


def spec_shard_phase_launch(args, stream_ptr):
    return int(lib.spec_shard_phase_launch(ctypes.byref(args), stream_ptr))


def spec_shard_decide_launch(args, stream_ptr):
    return int(lib.spec_shard_decide_launch(ctypes.byref(args), stream_ptr))


def spec_shard_draw_launch(args, stream_ptr):
    return int(lib.spec_shard_draw_launch(ctypes.byref(args), stream_ptr))


def spec_logprobs_workspace_bytes(B, R, V, top):
    if not _fits32(B, R, V, top):
        return 0  # (as for any invalid shape)
    return int(lib.spec_logprobs_workspace_bytes(int(B), int(R), int(V), int(top)))


def spec_logprobs_launch(args, stream_ptr):
    return int(lib.spec_logprobs_launch(ctypes.byref(args), stream_ptr))


def spec_kv_write_launch(args, stream_ptr):
    return int(lib.spec_kv_write_launch(ctypes.byref(args), stream_ptr))


def spec_kv_read_launch(args, stream_ptr):
    return int(lib.spec_kv_read_launch(ctypes.byref(args), stream_ptr))


def spec_attn_workspace_bytes(args):
    """Workspace of an attention from the sizes in its argument block."""
    return int(lib.spec_attn_workspace_bytes(ctypes.byref(args)))


def spec_attn_launch(args, stream_ptr):
    return int(lib.spec_attn_launch(ctypes.byref(args), stream_ptr))


def spec_status_string(status):
    return lib.spec_status_string(int(status)).decode()


# ------------------------------------------------------- torch conveniences
def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _logit_dtype(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError("logits must be bfloat16 or float32, got %s" % t.dtype)


def _check_dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")


def make_workspace(B, K, V, device="cuda"):
    """A workspace large enough for verifications of this shape (no
    initialisation needed; torch's allocations are 256-byte aligned)."""
    torch = _torch()
    n = spec_verify_workspace_bytes(B, K, V)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def verify_args(target, draft, draft_tokens, temperature, accepted, tokens, debug, workspace,
                seed=0, step=0, request_base=0, phase_event=None, phase_starts=0, draft_row_index=None,
                num_drafts=None, draft_stats=None):
    """Fill a SpecVerifyArgs from tensors (no copies).

    With draft_row_index [B, K] int32, draft is a 2-D [N, V] buffer (e.g. the
    drafter's logits) and draft row k of request b is its row
    draft_row_index[b, k].

    target [B or broadcast, K+1, V] and draft [B or broadcast, >=K, V] with a
    unit innermost stride; a request stride of 0 (expanded tensor) shares rows.
    """
    _check_dev(target, draft, draft_tokens, temperature, accepted, tokens, debug, workspace)
    B, K = draft_tokens.shape
    V = target.shape[-1]
    if target.stride(-1) != 1 or draft.stride(-1) != 1:
        raise ValueError("logits rows must be contiguous")
    if draft_tokens.dtype != _torch().int32 or not draft_tokens.is_contiguous():
        raise ValueError("draft_tokens must be contiguous int32 [B, K]")
    if temperature.dtype != _torch().float32 or not temperature.is_contiguous():
        raise ValueError("temperature must be contiguous float32 [B]")
    a = SpecVerifyArgs()
    a.B, a.K, a.V, a.dtype = B, K, V, _logit_dtype(target)
    if draft.dtype != target.dtype:
        raise TypeError("target and draft logits must share a dtype")
    a.target_logits = target.data_ptr()
    a.t_req_stride = target.stride(0) if target.shape[0] == B and B > 1 else 0
    a.t_row_stride = target.stride(1)
    a.draft_logits = draft.data_ptr()
    if draft_row_index is not None:
        _check_dev(draft_row_index)
        if draft.dim() != 2:
            raise ValueError("with a draft row table the draft logits are [N, V]")
        if draft_row_index.dtype != _torch().int32 or not draft_row_index.is_contiguous() or \
                tuple(draft_row_index.shape) != (B, K):
            raise ValueError("draft_row_index must be contiguous int32 [B, K]")
        a.d_req_stride, a.d_row_stride = 0, draft.stride(0)
        a.draft_row_index, a.draft_rows = draft_row_index.data_ptr(), draft.shape[0]
    else:
        a.d_req_stride = draft.stride(0) if draft.shape[0] == B and B > 1 else 0
        a.d_row_stride = draft.stride(1)
        a.draft_row_index, a.draft_rows = None, 0
    a.draft_tokens = draft_tokens.data_ptr()
    a.temperature = temperature.data_ptr()
    a.seed, a.step, a.request_base = int(seed) & (2 ** 64 - 1), int(step) & 0xFFFFFFFF, int(request_base)
    a.accepted_counts = accepted.data_ptr()
    a.output_tokens = tokens.data_ptr()
    a.debug_probs = debug.data_ptr() if debug is not None else None
    # workspace None: for spec_verify_launch_noalloc, which brings its own
    a.workspace = workspace.data_ptr() if workspace is not None else None
    a.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    a.phase_event = phase_event
    a.phase_starts = int(phase_starts)
    if num_drafts is not None:
        _check_dev(num_drafts)
        if num_drafts.dtype != _torch().int32 or not num_drafts.is_contiguous() or num_drafts.numel() != B:
            raise ValueError("num_drafts must be contiguous int32 [B]")
        a.num_drafts = num_drafts.data_ptr()
    else:
        a.num_drafts = None
    if draft_stats is not None:
        _check_dev(draft_stats)
        if draft_stats.numel() * draft_stats.element_size() < B * K * DRAFT_STATS_BYTES:
            raise ValueError("draft_stats must hold [B, K] records of %d bytes" % DRAFT_STATS_BYTES)
        a.draft_stats = draft_stats.data_ptr()
    else:
        a.draft_stats = None
    return a


def verify(target, draft, draft_tokens, temperature, seed=0, step=0, request_base=0, debug=False,
           workspace=None, stream=None, phase_starts=0, draft_row_index=None, num_drafts=None, draft_stats=None):
    """One verification step on torch's current stream.  Returns
    (accepted_counts [B] int32, output_tokens [B, K+1] int32, debug_probs
    [B, K, 2] float32 or None)."""
    torch = _torch()
    B, K = draft_tokens.shape
    V = target.shape[-1]
    dev = target.device
    accepted = torch.empty(B, dtype=torch.int32, device=dev)
    tokens = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
    dbg = torch.empty(B, K, 2, dtype=torch.float32, device=dev) if debug else None
    ws = workspace if workspace is not None else make_workspace(B, K, V, dev)
    a = verify_args(target, draft, draft_tokens, temperature, accepted, tokens, dbg, ws, seed, step,
                    request_base, phase_starts=phase_starts, draft_row_index=draft_row_index,
                    num_drafts=num_drafts, draft_stats=draft_stats)
    rc = spec_verify_launch(a, _stream_ptr(stream))
    if rc != SPEC_OK:
        raise SpecError(rc)
    return accepted, tokens, dbg


class ExpandOutputs:
    def __init__(self, **kw):
        self.__dict__.update(kw)


def expand_outputs(B, K, N_in, H, device, with_hidden=True, with_slots=False):
    torch = _torch()
    N_out = N_in + B * (K - 1)
    return ExpandOutputs(
        slot_mapping=torch.empty(N_out, dtype=torch.int64, device=device) if with_slots else None,
        out_token_ids=torch.empty(N_out, dtype=torch.int32, device=device),
        out_positions=torch.empty(N_out, dtype=torch.int64, device=device),
        rejected_mask=torch.empty(N_out, dtype=torch.uint8, device=device),
        masked_mask=torch.empty(N_out, dtype=torch.uint8, device=device),
        new_token_indices=torch.empty(B, K, dtype=torch.int32, device=device),
        hidden_map=torch.empty(N_in, dtype=torch.int32, device=device),
        out_start=torch.empty(B + 1, dtype=torch.int32, device=device),
        out_hidden=torch.empty(N_out, H, dtype=torch.bfloat16, device=device) if with_hidden else None)


def expand_args(in_token_ids, in_positions, in_start, accepted, bonus, K, mask_id, target_hidden,
                mask_hidden, out, verify_tokens=None, block_table=None, block_size=0):
    """bonus: [B] int32, or None with verify_tokens = the [B, K+1] output
    tokens of a verification (the bonus is then read at the accepted count).
    block_table: [B, max_blocks] int32 (row stride free, unit column stride)
    with block_size, when out.slot_mapping is given."""
    torch = _torch()
    _check_dev(in_token_ids, in_positions, in_start, accepted, bonus, target_hidden, mask_hidden)
    for t, dt in ((in_token_ids, torch.int32), (in_positions, torch.int64), (in_start, torch.int32),
                  (accepted, torch.int32), (bonus, torch.int32), (verify_tokens, torch.int32)):
        if t is not None and (t.dtype != dt or not t.is_contiguous()):
            raise ValueError("expected contiguous %s" % dt)
    a = SpecExpandArgs()
    B = accepted.shape[0]
    a.B, a.K, a.N_in, a.mask_token_id = B, int(K), in_token_ids.shape[0], int(mask_id)
    a.in_token_ids, a.in_positions, a.in_start = (in_token_ids.data_ptr(), in_positions.data_ptr(),
                                                   in_start.data_ptr())
    a.accepted_counts = accepted.data_ptr()
    a.bonus_tokens = bonus.data_ptr() if bonus is not None else None
    a.verify_output_tokens = verify_tokens.data_ptr() if verify_tokens is not None else None
    if out.out_hidden is not None:
        if target_hidden.dtype != torch.bfloat16 or target_hidden.stride(-1) != 1:
            raise ValueError("target_hidden must be bfloat16 with contiguous rows")
        a.H = target_hidden.shape[1]
        a.target_hidden = target_hidden.data_ptr()
        a.hidden_row_stride = target_hidden.stride(0)
        a.mask_hidden = mask_hidden.contiguous().data_ptr()
        a.out_hidden = out.out_hidden.data_ptr()
    else:
        a.H, a.target_hidden, a.hidden_row_stride, a.mask_hidden, a.out_hidden = 0, None, 0, None, None
    if getattr(out, "slot_mapping", None) is not None:
        if block_table is None or block_table.dtype != torch.int32 or block_table.stride(-1) != 1:
            raise ValueError("slot mapping needs an int32 block table with unit column stride")
        _check_dev(block_table)
        a.block_table = block_table.data_ptr()
        a.bt_row_stride = block_table.stride(0)
        a.max_blocks = block_table.shape[1]
        a.block_size = int(block_size)
        a.slot_mapping = out.slot_mapping.data_ptr()
    else:
        a.block_table, a.bt_row_stride, a.max_blocks, a.block_size, a.slot_mapping = None, 0, 0, 0, None
    a.out_token_ids, a.out_positions = out.out_token_ids.data_ptr(), out.out_positions.data_ptr()
    a.rejected_mask, a.masked_mask = out.rejected_mask.data_ptr(), out.masked_mask.data_ptr()
    a.new_token_indices, a.hidden_map = out.new_token_indices.data_ptr(), out.hidden_map.data_ptr()
    a.out_start = out.out_start.data_ptr()
    return a


def expand(in_token_ids, in_positions, in_start, accepted, bonus, K, mask_id, target_hidden=None,
           mask_hidden=None, stream=None, out=None, verify_tokens=None, block_table=None, block_size=0):
    """One expansion on torch's current stream; returns an ExpandOutputs
    (with slot_mapping when a block table is given)."""
    B = accepted.shape[0]
    H = target_hidden.shape[1] if target_hidden is not None else 0
    if out is None:
        out = expand_outputs(B, K, in_token_ids.shape[0], H, accepted.device,
                             with_hidden=target_hidden is not None, with_slots=block_table is not None)
    a = expand_args(in_token_ids, in_positions, in_start, accepted, bonus, K, mask_id, target_hidden,
                    mask_hidden, out, verify_tokens, block_table=block_table, block_size=block_size)
    rc = spec_expand_launch(a, _stream_ptr(stream))
    if rc != SPEC_OK:
        raise SpecError(rc)
    return out


# ------------------------------------------------------------ draft sampling
def draft_args(logits, row_index, temperature, tokens, workspace, seed=0, step=0, request_base=0, stats_out=None):
    """Fill a SpecDraftArgs: logits [N, V] (unit column stride), row_index
    [B, K] int32, temperature [B] float32, tokens [B, K] int32 out."""
    torch = _torch()
    _check_dev(logits, row_index, temperature, tokens, workspace)
    if logits.dim() != 2 or logits.stride(-1) != 1:
        raise ValueError("logits must be [N, V] with contiguous rows")
    for t, dt in ((row_index, torch.int32), (temperature, torch.float32), (tokens, torch.int32)):
        if t.dtype != dt or not t.is_contiguous():
            raise ValueError("expected contiguous %s" % dt)
    a = SpecDraftArgs()
    B, K = row_index.shape
    a.B, a.K, a.V, a.N, a.dtype = B, K, logits.shape[1], logits.shape[0], _logit_dtype(logits)
    a.logits, a.row_stride = logits.data_ptr(), logits.stride(0)
    a.row_index, a.temperature, a.tokens = row_index.data_ptr(), temperature.data_ptr(), tokens.data_ptr()
    a.seed, a.step, a.request_base = int(seed) & (2 ** 64 - 1), int(step) & 0xFFFFFFFF, int(request_base)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    if stats_out is not None:
        _check_dev(stats_out)
        if stats_out.numel() * stats_out.element_size() < B * K * DRAFT_STATS_BYTES:
            raise ValueError("stats_out must hold [B, K] records of %d bytes" % DRAFT_STATS_BYTES)
        a.stats_out = stats_out.data_ptr()
    else:
        a.stats_out = None
    return a


def draft_stats_buffer(B, K, device="cuda"):
    """Device memory for the [B, K] draft statistics records."""
    return _torch().empty(B * K * DRAFT_STATS_BYTES, dtype=_torch().uint8, device=device)


def draft_sample(logits, row_index, temperature, seed=0, step=0, request_base=0, workspace=None, stream=None,
                 stats_out=None):
    """Draft tokens [B, K] int32 sampled at rows row_index of logits, on
    torch's current stream (and, with stats_out, the rows' statistics for
    the verification of these tokens)."""
    torch = _torch()
    B, K = row_index.shape
    dev = logits.device
    tokens = torch.empty(B, K, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(spec_draft_workspace_bytes(B, K, logits.shape[1]), 16), dtype=torch.uint8,
                                device=dev)
    a = draft_args(logits, row_index, temperature, tokens, workspace, seed, step, request_base, stats_out)
    rc = spec_draft_sample_launch(a, _stream_ptr(stream))
    if rc != SPEC_OK:
        raise SpecError(rc)
    return tokens


# ---------------------------------------------------- vocab-sharded verify
SHARD_RECORD_BYTES = 32


def phase_count(K, phase_starts):
    """Phases of a phase_starts cut of positions 0..K (1 for one pass)."""
    return 1 + sum(1 for k in range(1, int(K) + 1) if (int(phase_starts) >> k) & 1)


class ShardSetup:
    """Argument blocks of the G shards of one vocab-sharded verification and
    the arrays they exchange (records, masses) and write (per-shard accepted
    counts [G, B], output tokens [G, B, K+1])."""

    def __init__(self, shards, records, masses, acc, tok, stream_ptr, phases=1):
        self.shards, self.records, self.masses = shards, records, masses
        self.acc, self.tok, self.stream_ptr = acc, tok, stream_ptr
        self.phases = phases

    def launch(self, stage, h, phase=0):
        """Enqueue stage 0 (statistics of a phase), 1 (decisions), 2 (draw)
        or 3 (the accept tests of a phase before the last) of shard h."""
        launch = (spec_shard_stats_launch, spec_shard_decide_launch, spec_shard_draw_launch,
                  spec_shard_phase_launch)[stage]
        a = self.shards[h][0]
        a.phase = int(phase)
        rc = launch(a, self.stream_ptr)
        if rc != SPEC_OK:
            raise SpecError(rc)

    def schedule(self):
        """The (stage, phase) launches of one verification in order; each is
        run on every shard before the next (an exchange between them)."""
        out = []
        for p in range(self.phases):
            out.append((0, p))
            if p + 1 < self.phases:
                out.append((3, p))
        return out + [(1, 0), (2, 0)]

    def run(self):
        """Every stage of every shard, in stage order (the exchanges between
        stages are the shared arrays)."""
        for stage, p in self.schedule():
            for h in range(len(self.shards)):
                self.launch(stage, h, p)


def shard_setup(target, draft, draft_tokens, temperature, G, seed=0, step=0, request_base=0, bounds=None,
                stream=None, phase_starts=0, num_drafts=None, draft_row_index=None):
    """The argument blocks of a verification with the vocabulary split over G
    shards (bounds: G+1 slice boundaries, default as equal as possible), each
    shard reading only its slice of the logits, with their workspaces and
    exchange arrays allocated here.  With draft_row_index [B, K] int32, draft
    is a 2-D [N, V] buffer of draft rows (each shard reads its slice of
    them); num_drafts [B] int32: ragged draft counts; phase_starts: early
    exit as for verify()."""
    torch = _torch()
    B, K = draft_tokens.shape
    V = target.shape[-1]
    dev = target.device
    if bounds is None:
        bounds = [(V * h) // G for h in range(G + 1)]
    if len(bounds) != G + 1 or bounds[0] != 0 or bounds[-1] != V:
        raise ValueError("bounds must run from 0 to V in G steps")
    R = 2 * K + 1
    records = torch.empty(G * B * R * SHARD_RECORD_BYTES, dtype=torch.uint8, device=dev)
    masses = torch.empty(G * B * 2, dtype=torch.float64, device=dev)
    acc = torch.empty(G, B, dtype=torch.int32, device=dev)
    tok = torch.empty(G, B, K + 1, dtype=torch.int32, device=dev)
    shards = []
    for h in range(G):
        v0, v1 = bounds[h], bounds[h + 1]
        ws = torch.empty(max(spec_shard_workspace_bytes(B, K, v1 - v0), 16), dtype=torch.uint8, device=dev)
        t, d = target[..., v0:v1], draft[..., v0:v1]
        a = SpecShardArgs()
        a.B, a.K, a.V, a.dtype, a.G, a.g, a.v0, a.Vs = B, K, V, _logit_dtype(target), G, h, v0, v1 - v0
        a.target_logits = t.data_ptr()
        a.t_req_stride = target.stride(0) if target.shape[0] == B and B > 1 else 0
        a.t_row_stride = target.stride(1)
        a.draft_logits = d.data_ptr()
        a.d_req_stride = draft.stride(0) if draft.shape[0] == B and B > 1 else 0
        a.d_row_stride = draft.stride(1)
        a.draft_tokens, a.temperature = draft_tokens.data_ptr(), temperature.data_ptr()
        a.seed, a.step, a.request_base = int(seed) & (2 ** 64 - 1), int(step) & 0xFFFFFFFF, int(request_base)
        a.records, a.masses = records.data_ptr(), masses.data_ptr()
        a.accepted_counts, a.output_tokens = acc[h].data_ptr(), tok[h].data_ptr()
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
        if draft_row_index is not None:
            a.d_req_stride, a.d_row_stride = 0, draft.stride(0)
            a.draft_row_index, a.draft_rows = draft_row_index.data_ptr(), draft.shape[0]
        else:
            a.draft_row_index, a.draft_rows = None, 0
        a.num_drafts = num_drafts.data_ptr() if num_drafts is not None else None
        a.phase_starts, a.phase = int(phase_starts), 0
        shards.append((a, ws))
    return ShardSetup(shards, records, masses, acc, tok, _stream_ptr(stream), phase_count(K, phase_starts))


def verify_sharded(target, draft, draft_tokens, temperature, G, seed=0, step=0, request_base=0, bounds=None,
                   stream=None, phase_starts=0, num_drafts=None, draft_row_index=None):
    """The verification with the vocabulary split over G shards, each stage of
    each shard launched through the C ABI on one GPU; the exchanges between
    shards are the shared record and mass arrays, and the last one (the
    sampled token, -1 on every shard but its owner) an element-wise maximum.
    bounds: G+1 slice boundaries (default: as equal as possible).  Returns
    (accepted [B], output_tokens [B, K+1], per-shard accepted counts [G, B])."""
    st = shard_setup(target, draft, draft_tokens, temperature, G, seed=seed, step=step, request_base=request_base,
                     bounds=bounds, stream=stream, phase_starts=phase_starts, num_drafts=num_drafts,
                     draft_row_index=draft_row_index)
    st.run()
    return st.acc[0].clone(), st.tok.max(dim=0).values, st.acc


# --------------------------------- operators around a verification step
# (kept short on the host: at the sizes of one decode step these calls cost
# about what their kernels do)
class _on:
    """Device `dev` current, and `stream` (or that device's current
    stream) its current stream: what is allocated here belongs to the stream
    that the work is enqueued on."""
    __slots__ = ("ptr", "ctx")

    def __init__(self, dev, stream=None):
        torch = _torch()
        self.ctx = None
        if stream is None:
            # (the address alone: a torch.cuda.Stream object costs a quarter of a small call)
            self.ptr = torch._C._cuda_getCurrentRawStream(dev.index)
            if torch._C._cuda_getDevice() != dev.index:
                self.ctx = torch.cuda.device(dev)
        else:
            if stream.device != dev:
                raise ValueError("the stream is on another device than the tensors")
            self.ctx = torch.cuda.stream(stream)
            self.ptr = stream.cuda_stream

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _fits32(*sizes):
    return max(sizes) <= 0x7fffffff and min(sizes) >= -0x80000000


def _int32(*sizes):
    """The library counts in 32 bits, and ctypes drops what is above them."""
    if not _fits32(*sizes):
        raise ValueError("a size past 32 bits among %s" % list(sizes))


def _gpu_device(t):
    if not t.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    return t.device


def _want(t, dtype, shape, dev, name):
    """The address of a contiguous tensor of this type, shape and device."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s %s" % (name, dtype, list(shape)))
    if t.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    return t.data_ptr()


def _want_workspace(t, dev):
    if t is None:
        return None, 0
    if t.device != dev or not t.is_contiguous():
        raise ValueError("the workspace must be contiguous on the tensors' GPU")
    return t.data_ptr(), t.numel() * t.element_size()


# ------------------------------------------------- token log probabilities
class TokenLogprobs:
    """logprobs [B, R] and entropy [B, R] float32 (entropy None if not asked
    for), top_ids [B, R, top] int32, top_logprobs [B, R, top] float32."""
    __slots__ = ("logprobs", "entropy", "top_ids", "top_logprobs")

    def __init__(self, logprobs, entropy, top_ids, top_logprobs):
        self.logprobs, self.entropy, self.top_ids, self.top_logprobs = logprobs, entropy, top_ids, top_logprobs


def token_logprobs_outputs(B, R, top, device, entropy=True):
    torch = _torch()
    f32, empty = torch.float32, torch.empty
    return TokenLogprobs(empty((B, R), dtype=f32, device=device),
                         empty((B, R), dtype=f32, device=device) if entropy else None,
                         empty((B, R, top), dtype=torch.int32, device=device),
                         empty((B, R, top), dtype=f32, device=device))


def token_logprobs_args(logits, tokens, temperature, out, workspace):
    """Fill a SpecLogprobsArgs (no copies): logits [B, R, V] with unit column
    stride (an expanded request dimension shares rows), tokens [B, R] int32,
    temperature [B] float32 or None, out a TokenLogprobs."""
    torch = _torch()
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V]")
    _int32(*logits.shape)
    dev = _gpu_device(logits)
    B, R, _ = logits.shape
    if out.entropy is not None:
        _want(out.entropy, torch.float32, (B, R), dev, "entropy")
    top = out.top_ids.shape[-1]
    _want(out.logprobs, torch.float32, (B, R), dev, "logprobs")
    _want(out.top_ids, torch.int32, (B, R, top), dev, "top_ids")
    _want(out.top_logprobs, torch.float32, (B, R, top), dev, "top_logprobs")
    return _logprobs_args(logits, tokens, temperature, top, out, _want_workspace(workspace, dev))


def _logprobs_args(logits, tokens, temperature, top, out, ws):
    torch = _torch()
    dev = logits.device
    B, R, V = logits.shape
    s0, s1, s2 = logits.stride()
    if s2 != 1 and V > 1:
        raise ValueError("logits must be [B, R, V] with contiguous rows")
    return SpecLogprobsArgs(
        B, R, V, _logit_dtype(logits), logits.data_ptr(), s0 if B > 1 else 0, s1 if R > 1 else V,
        _want(tokens, torch.int32, (B, R), dev, "tokens"),
        None if temperature is None else _want(temperature, torch.float32, (B,), dev, "temperature"), top,
        out.logprobs.data_ptr(), None if out.entropy is None else out.entropy.data_ptr(), out.top_ids.data_ptr(),
        out.top_logprobs.data_ptr(), ws[0], ws[1])


def token_logprobs(logits, tokens, temperature=None, top=0, entropy=True, workspace=None, stream=None, out=None):
    """Log probabilities of tokens [B, R] (int32; -1: no token, its row is not
    read) under softmax(logits / T), logits [B, R, V]; the entropy of each row
    and its `top` most likely tokens.  tokens may be the output_tokens of a
    verification with logits its target.  Enqueued on `stream` or the tensors'
    device's current stream; returns a TokenLogprobs (`out`, where given, says
    with its shapes what is computed)."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V]")
    B, R, V = logits.shape
    if (B | R | V) > 0x7fffffff:
        _int32(B, R, V)
    dev = _gpu_device(logits)
    if not 0 <= top <= SPEC_MAX_TOP:
        raise ValueError("top must be in 0..%d" % SPEC_MAX_TOP)
    with _on(dev, stream) as s:
        if out is not None:
            top = out.top_ids.shape[-1]
        if workspace is None:
            torch = _torch()
            workspace = torch.empty(max(lib.spec_logprobs_workspace_bytes(B, R, V, top), 16), dtype=torch.uint8,
                                    device=dev)
        if out is not None:
            a = token_logprobs_args(logits, tokens, temperature, out, workspace)
        else:
            out = token_logprobs_outputs(B, R, top, dev, entropy)
            a = _logprobs_args(logits, tokens, temperature, top, out, _want_workspace(workspace, dev))
        rc = lib.spec_logprobs_launch(a, s)
    if rc != SPEC_OK:
        raise SpecError(rc)
    return out


# ----------------------------------------------------- 8-bit paged KV cache
class KVCache:
    """A paged cache of keys and values in 8 bits: codes k, v (uint8, or
    float8_e4m3fn) [num_blocks, block_size, heads, head_dim] and scale
    exponents k_scale, v_scale (uint8, or float8_e8m0fnu) [num_blocks, heads,
    block_size / scale_tokens]; the value of a code is code * 2^(byte - 127).
    Blocks may hold their heads outside their tokens (a transposed view); k
    and v share strides, and so do their scales.  block_size is a power of two
    from 16 to 1024, scale_tokens one from 1 to 64, head_dim a multiple of 16
    up to 256."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "num_blocks", "block_size", "heads", "head_dim", "scale_tokens",
                 "device", "args")

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or k_scale.dim() != 3:
            raise ValueError("codes must be [num_blocks, block_size, heads, head_dim], scales [num_blocks, heads, "
                             "groups]")
        torch = _torch()
        if k.dtype not in (torch.uint8, torch.float8_e4m3fn) or v.dtype != k.dtype or \
                k_scale.dtype not in (torch.uint8, torch.float8_e8m0fnu) or v_scale.dtype != k_scale.dtype:
            raise TypeError("codes must be uint8 or float8_e4m3fn, scales uint8 or float8_e8m0fnu, alike for k and v")
        _int32(*k.shape)
        dev = _gpu_device(k)
        if v.device != dev or k_scale.device != dev or v_scale.device != dev:
            raise ValueError("all tensors must be on the same GPU")
        nb, bs, heads, dim = k.shape
        snb, sheads, groups = k_scale.shape
        st, sst = k.stride(), k_scale.stride()
        if v.shape != k.shape or v.stride() != st or v_scale.shape != k_scale.shape or v_scale.stride() != sst or \
                snb != nb or sheads != heads:
            raise ValueError("k and v (and their scales) must agree in shape and strides")
        if st[3] != 1 or (groups > 1 and sst[2] != 1) or groups < 1 or bs % groups:
            raise ValueError("codes must be contiguous along head_dim, scales along their groups, which divide a block")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_blocks, self.block_size, self.heads, self.head_dim = nb, bs, heads, dim
        self.scale_tokens, self.device = bs // groups, dev
        self.args = SpecKVCache(nb, bs, bs // groups, heads, dim, k.data_ptr(), v.data_ptr(), st[0], st[1],
                                st[2] if heads > 1 else dim, k_scale.data_ptr(), v_scale.data_ptr(), sst[0],
                                sst[1] if heads > 1 else groups)


def make_kv_cache(num_blocks, block_size, heads, head_dim, scale_tokens=None, device="cuda"):
    """A KVCache of zeros; scale_tokens tokens share a scale (default: a whole
    block, at most 64)."""
    torch = _torch()
    st = min(block_size, 64) if scale_tokens is None else scale_tokens
    if st < 1 or block_size % st:
        raise ValueError("scale_tokens must divide block_size")
    codes = [torch.zeros(num_blocks, block_size, heads, head_dim, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros(num_blocks, heads, block_size // st, dtype=torch.uint8, device=device) for _ in range(2)]
    return KVCache(*codes, *scales)


def _kv_dtype(dtype):
    torch = _torch()
    if dtype == torch.bfloat16:
        return SPEC_BF16
    if dtype == torch.float32:
        return SPEC_F32
    raise TypeError("keys and values must be bfloat16 or float32, got %s" % dtype)


def kv_write_args(cache, key, value, slots):
    """Fill a SpecKVWriteArgs (no copies): key and value [N, heads, head_dim]
    with unit stride along head_dim, slots [N] int64 (-1: not written)."""
    N, dev = slots.shape[0], cache.device
    if N > 0x7fffffff:
        _int32(N)
    shape = (N, cache.heads, cache.head_dim)
    k0, k1, k2 = key.stride() if key.dim() == 3 else (0, 0, 0)
    v0, v1, v2 = value.stride() if value.dim() == 3 else (0, 0, 0)
    if key.shape != shape or value.shape != shape or k2 != 1 or v2 != 1:
        raise ValueError("key and value must be [N, heads, head_dim], contiguous along head_dim")
    if key.dtype != value.dtype:
        raise TypeError("key and value must share a dtype")
    if key.device != dev or value.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    return SpecKVWriteArgs(cache.args, N, _kv_dtype(key.dtype), key.data_ptr(), value.data_ptr(), k0, k1, v0, v1,
                           _want(slots, _torch().int64, (N,), dev, "slots"))


def kv_write(cache, key, value, slots, stream=None):
    """Quantise keys and values [N, heads, head_dim] into the cache at slots
    [N] int64 (the slot_mapping of an expansion; -1 is skipped); returns the
    cache."""
    with _on(cache.device, stream) as s:
        rc = lib.spec_kv_write_launch(kv_write_args(cache, key, value, slots), s)
    if rc != SPEC_OK:
        raise SpecError(rc)
    return cache


def kv_read(cache, slots, dtype=None, stream=None, out=None):
    """Keys and values [N, heads, head_dim] at slots [N] int64, bfloat16 (the
    default) or float32, zeros where a slot is -1."""
    torch = _torch()
    N, dev = slots.shape[0], cache.device
    if N > 0x7fffffff:
        _int32(N)
    shape = (N, cache.heads, cache.head_dim)
    with _on(cache.device, stream) as s:
        if out is None:
            dt = torch.bfloat16 if dtype is None else dtype
            key, value = torch.empty(shape, dtype=dt, device=dev), torch.empty(shape, dtype=dt, device=dev)
        else:
            key, value = out
            dt = key.dtype if dtype is None else dtype
            _want(key, dt, shape, dev, "key")
            _want(value, dt, shape, dev, "value")
        a = SpecKVReadArgs(cache.args, N, _kv_dtype(dt), key.data_ptr(), value.data_ptr(),
                           _want(slots, torch.int64, (N,), dev, "slots"))
        rc = lib.spec_kv_read_launch(a, s)
    if rc != SPEC_OK:
        raise SpecError(rc)
    return key, value


def kv_attention_args(q, cache, block_table, q_start, ctx_len, max_q, max_ctx, scale, out, lse=None, window=0,
                      sinks=None, workspace=None):
    """Fill a SpecAttnArgs (no copies): q [N, q_heads, head_dim] bfloat16 with
    unit stride along head_dim, block_table [B, max_blocks] int32 (row stride
    free), q_start [B + 1] and ctx_len [B] int32, sinks [q_heads] float32,
    out [N, q_heads, head_dim] bfloat16, lse [N, q_heads] float32."""
    torch = _torch()
    dev = cache.device
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.stride(2) != 1:
        raise ValueError("q must be [N, q_heads, head_dim], contiguous along head_dim")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16, got %s" % q.dtype)
    N, Hq, D = q.shape
    B = ctx_len.shape[0]
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B or \
            (block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("block_table must be int32 [B, max_blocks] with unit column stride")
    if q.device != dev or block_table.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    max_blocks = block_table.shape[1]
    if not 0 <= (B | N | Hq | max_q | max_ctx | window | max_blocks) <= 0x7fffffff:  # (some bit above the 31, or a sign)
        _int32(B, N, Hq, max_q, max_ctx, window, max_blocks)
    ws = _want_workspace(workspace, dev)
    return SpecAttnArgs(
        cache.args, B, N, Hq, max_q, max_ctx, window, SPEC_BF16, scale, q.data_ptr(), q.stride(0), q.stride(1),
        _want(q_start, torch.int32, (B + 1,), dev, "q_start"), _want(ctx_len, torch.int32, (B,), dev, "ctx_len"),
        block_table.data_ptr(), block_table.stride(0) if B > 1 else max_blocks, max_blocks,
        None if sinks is None else _want(sinks, torch.float32, (Hq,), dev, "sinks"),
        _want(out, torch.bfloat16, (N, Hq, D), dev, "out"),
        None if lse is None else _want(lse, torch.float32, (N, Hq), dev, "lse"), ws[0], ws[1])


def kv_attention(q, cache, block_table, q_start, ctx_len, max_q, max_ctx=None, scale=None, window=0, sinks=None,
                 return_lse=False, workspace=None, stream=None, out=None):
    """Attention of the new tokens q [N, q_heads, head_dim] of B requests
    (request b: rows q_start[b]..q_start[b+1] - 1) over their cached contexts
    of ctx_len[b] tokens, the new ones included and last.  max_q and max_ctx
    bound the new tokens and the context of a request (max_ctx defaults to
    what the block table holds); scale defaults to head_dim ** -0.5; window >
    0 sees only the last `window` positions; sinks [q_heads] float32 take part
    in the softmax without a value.  Returns (out, lse or None); rows of `out`
    and lse outside every request's range are not written."""
    torch = _torch()
    dev = cache.device
    if max_ctx is None:
        max_ctx = min(block_table.shape[-1] * cache.block_size, 1 << 30)
    if scale is None:
        scale = cache.head_dim ** -0.5
    with _on(cache.device, stream) as s:
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if return_lse else None
        a = kv_attention_args(q, cache, block_table, q_start, ctx_len, max_q, max_ctx, scale, out, lse, window, sinks,
                              workspace)
        if workspace is None:
            n = lib.spec_attn_workspace_bytes(a)
            if n:
                workspace = torch.empty(n, dtype=torch.uint8, device=dev)
                a.workspace, a.workspace_bytes = workspace.data_ptr(), n
        rc = lib.spec_attn_launch(a, s)
    if rc != SPEC_OK:
        raise SpecError(rc)
    return out, lse
