"""ctypes binding of libspecverify.so.

Argument marshalling only: every step of the verify computation runs in the
library's HIP kernels.  PyTorch provides device memory and the current
stream.  There is no fallback: when the library is missing or no GPU is
present, the calls raise.
"""

import contextlib
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_F32, SV_BF16, SV_F16 = 0, 1, 2
MAX_NODES = 64
PROBE_POS, PROBE_ROW = 8, 4
STATUS = {0: "SV_OK", -1: "SV_EINVAL", -2: "SV_ESHAPE", -3: "SV_EDTYPE", -4: "SV_EHIP", -5: "SV_ENOMEM",
          -6: "SV_EALIGN", -7: "SV_ECAPTURE", -8: "SV_ETOOBIG"}
KERNEL_KINDS = ("stats", "topp", "rows", "smc", "produce", "tree_attention", "tree_join", "verify_clear",
                "tree_verify", "cache_plan", "cache_copy", "latent_attention", "latent_join",
                "head_product", "prompt_plan", "prompt_expand", "prompt_scale", "prompt_attention", "beam_stats",
                "beam_select", "beam_reorder", "reserve_plan", "reserve_write", "cache_write")

EXPORTS = ("spec_verify", "spec_verify_noalloc", "spec_verify_probe", "spec_greedy_verify", "spec_hispec_verify", "spec_smc_step",
           "spec_draft_produce",
           "spec_tree_attention", "spec_tree_attention_workspace", "spec_verify_tree", "spec_verify_tree_workspace",
           "spec_cache_commit", "spec_cache_fork", "spec_cache_workspace",
           "spec_latent_attention", "spec_latent_attention_workspace", "spec_head_product", "spec_latent_prompt",
           "spec_latent_prompt_workspace", "spec_cache_reserve", "spec_cache_reserve_workspace", "spec_cache_write",
           "spec_beam_select", "spec_beam_workspace", "spec_beam_reorder",
           "spec_verify_strerror",
           "spec_verify_release",
           "spec_verify_abi_version", "spec_verify_profile_enable", "spec_verify_profile_read",
           "spec_verify_stream_read")


class SvLogits(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32),
        ("P", ctypes.c_int32),
        ("V", ctypes.c_int32),
        ("stride_b", ctypes.c_int64),
        ("stride_p", ctypes.c_int64),
    ]


class SvTreeAttention(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("q", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64 * 3),
        ("k_tree", ctypes.c_void_p),
        ("v_tree", ctypes.c_void_p),
        ("k_tree_stride", ctypes.c_int64 * 3),
        ("v_tree_stride", ctypes.c_int64 * 3),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("k_cache_stride", ctypes.c_int64 * 3),
        ("v_cache_stride", ctypes.c_int64 * 3),
        ("pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64),
        ("len", ctypes.c_void_p),
        ("parent", ctypes.c_void_p),
        ("n_nodes", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("sinks", ctypes.c_int32),
        ("out", ctypes.c_void_p),
        ("out_stride", ctypes.c_int64 * 3),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_int64),
    ]


class SvCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("layers", ctypes.c_int32),
        ("pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("k_stride", ctypes.c_int64 * 4),
        ("v_stride", ctypes.c_int64 * 4),
        ("table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64),
        ("len", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("width", ctypes.c_int32),
    ]


class SpecVerifyError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def load(path=LIB_PATH):
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m rejection_sampling_verifier_amd.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.spec_verify.argtypes = [P(SvLogits), P(SvLogits), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                ctypes.c_float, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.spec_verify.restype = ctypes.c_int
    lib.spec_verify_noalloc.argtypes = lib.spec_verify.argtypes
    lib.spec_verify_noalloc.restype = ctypes.c_int
    lib.spec_verify_probe.argtypes = lib.spec_verify.argtypes[:9] + [ctypes.c_void_p] * 3
    lib.spec_verify_probe.restype = ctypes.c_int
    lib.spec_greedy_verify.argtypes = [P(SvLogits), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32] + \
        [ctypes.c_void_p] * 4
    lib.spec_greedy_verify.restype = ctypes.c_int
    lib.spec_hispec_verify.argtypes = [P(SvLogits)] * 3 + [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                                            ctypes.c_float, ctypes.c_uint64] + [ctypes.c_void_p] * 4
    lib.spec_hispec_verify.restype = ctypes.c_int
    lib.spec_smc_step.argtypes = [P(SvLogits), P(SvLogits), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                  ctypes.c_double, ctypes.c_uint64] + [ctypes.c_void_p] * 6
    lib.spec_smc_step.restype = ctypes.c_int
    lib.spec_draft_produce.argtypes = [P(SvLogits), ctypes.c_int32, ctypes.c_uint64, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]
    lib.spec_draft_produce.restype = ctypes.c_int
    vp = ctypes.c_void_p
    lib.spec_tree_attention.argtypes = [P(SvTreeAttention), vp]
    lib.spec_tree_attention.restype = ctypes.c_int
    lib.spec_tree_attention_workspace.argtypes = [P(SvTreeAttention)]
    lib.spec_tree_attention_workspace.restype = ctypes.c_int64
    lib.spec_verify_tree.argtypes = [P(SvLogits), P(SvLogits)] + [vp] * 9 + [ctypes.c_int64, vp]
    lib.spec_verify_tree.restype = ctypes.c_int
    lib.spec_verify_tree_workspace.argtypes = [ctypes.c_int32] * 5
    lib.spec_verify_tree_workspace.restype = ctypes.c_int64
    i64x4 = ctypes.c_int64 * 4
    lib.spec_cache_commit.argtypes = [P(SvCache), vp, vp, i64x4, i64x4, ctypes.c_int32, vp, vp, vp, ctypes.c_int64, vp,
                                      vp, vp, ctypes.c_int64, vp]
    lib.spec_cache_commit.restype = ctypes.c_int
    lib.spec_cache_fork.argtypes = [P(SvCache), vp, vp, ctypes.c_int64, vp, vp, vp, ctypes.c_int64, vp]
    lib.spec_cache_fork.restype = ctypes.c_int
    lib.spec_cache_workspace.argtypes = [ctypes.c_int32] * 3
    lib.spec_cache_workspace.restype = ctypes.c_int64
    lib.spec_verify_strerror.argtypes = [ctypes.c_int]
    lib.spec_verify_strerror.restype = ctypes.c_char_p
    lib.spec_verify_release.argtypes = []
    lib.spec_verify_release.restype = None
    lib.spec_verify_abi_version.argtypes = []
    lib.spec_verify_abi_version.restype = ctypes.c_int
    lib.spec_verify_profile_enable.argtypes = [ctypes.c_int]
    lib.spec_verify_profile_enable.restype = ctypes.c_int
    lib.spec_verify_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int]
    lib.spec_verify_profile_read.restype = ctypes.c_int
    lib.spec_verify_stream_read.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
                                            ctypes.c_void_p]
    lib.spec_verify_stream_read.restype = ctypes.c_int
    _lib = lib
    return lib


def _desc(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [B, P, V]")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous along V")
    if t.dtype == torch.float32:
        dt = SV_F32
    elif t.dtype == torch.bfloat16:
        dt = SV_BF16
    else:
        raise ValueError(f"{name}: dtype {t.dtype} is not float32 or bfloat16")
    B, P, V = t.shape
    return SvLogits(t.data_ptr(), dt, B, P, V, t.stride(0), t.stride(1))


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(lib, rc):
    if rc < 0:
        raise SpecVerifyError(rc, lib.spec_verify_strerror(rc).decode())


def verify(target, draft, draft_tokens, draft_len=None, temperature=1.0, top_p=1.0, seed=0, *, stream=None,
           out_tokens=None, out_n_accepted=None, probe=False, noalloc=False):
    """The verify step on device tensors.

    target [B, K+1, V] and draft [B, K, V]: bfloat16 or float32, V contiguous.
    draft_tokens [B, K] int32 contiguous; draft_len [B] int32 or None.
    Returns (tokens [B, K+1] int32, n_accepted [B] int32), plus
    (probe_pos [B, K+1, 8], probe_row [B, 4]) float64 when probe is set.
    noalloc: call spec_verify_noalloc (no device allocation by the library;
    the caller passes out_tokens and out_n_accepted to allocate nothing at
    all).
    """
    lib = load()
    if draft_tokens.dtype != torch.int32 or not draft_tokens.is_contiguous():
        raise ValueError("draft_tokens must be contiguous int32")
    if draft_len is not None and (draft_len.dtype != torch.int32 or not draft_len.is_contiguous()):
        raise ValueError("draft_len must be contiguous int32")
    if noalloc and probe:
        raise ValueError("the no-allocation entry point has no probe")
    dev = target.device
    B, K1 = target.shape[0], target.shape[1]
    if out_tokens is None:
        out_tokens = torch.empty((B, K1), dtype=torch.int32, device=dev)
    if out_n_accepted is None:
        out_n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    td, dd = _desc(target, "target"), _desc(draft, "draft")
    args = [ctypes.byref(td), ctypes.byref(dd), ctypes.c_void_p(draft_tokens.data_ptr()),
            ctypes.c_void_p(draft_len.data_ptr() if draft_len is not None else None),
            ctypes.c_float(temperature), ctypes.c_float(top_p), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
            ctypes.c_void_p(out_tokens.data_ptr()), ctypes.c_void_p(out_n_accepted.data_ptr())]
    sh = _stream_handle(stream, dev)
    if probe:
        pp = torch.empty((B, K1, PROBE_POS), dtype=torch.float64, device=dev)
        pr = torch.empty((B, PROBE_ROW), dtype=torch.float64, device=dev)
        _check(lib, lib.spec_verify_probe(*args, ctypes.c_void_p(pp.data_ptr()), ctypes.c_void_p(pr.data_ptr()), sh))
        return out_tokens, out_n_accepted, pp, pr
    if noalloc:
        _check(lib, lib.spec_verify_noalloc(*args, sh))
    else:
        _check(lib, lib.spec_verify(*args, sh))
    return out_tokens, out_n_accepted


def greedy_verify(target, draft_tokens, draft_len=None, k=0, *, stream=None, out_tokens=None, out_n_accepted=None,
                  out_topk=None):
    """Greedy verify on device tensors: target [B, K+1, V] (bfloat16 or
    float32, V contiguous), draft_tokens [B, K] int32.  Returns (tokens
    [B, K+1] int32, n_accepted [B] int32, topk [B, k] int32)."""
    lib = load()
    if draft_tokens.dtype != torch.int32 or not draft_tokens.is_contiguous():
        raise ValueError("draft_tokens must be contiguous int32")
    if draft_len is not None and (draft_len.dtype != torch.int32 or not draft_len.is_contiguous()):
        raise ValueError("draft_len must be contiguous int32")
    dev = target.device
    B, K1 = target.shape[0], target.shape[1]
    if out_tokens is None:
        out_tokens = torch.empty((B, K1), dtype=torch.int32, device=dev)
    if out_n_accepted is None:
        out_n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_topk is None:
        out_topk = torch.empty((B, max(k, 1)), dtype=torch.int32, device=dev)
    td = _desc(target, "target")
    _check(lib, lib.spec_greedy_verify(ctypes.byref(td), ctypes.c_void_p(draft_tokens.data_ptr()),
                                       ctypes.c_void_p(draft_len.data_ptr() if draft_len is not None else None),
                                       ctypes.c_int32(k), ctypes.c_void_p(out_tokens.data_ptr()),
                                       ctypes.c_void_p(out_n_accepted.data_ptr()),
                                       ctypes.c_void_p(out_topk.data_ptr()), _stream_handle(stream, dev)))
    return out_tokens, out_n_accepted, out_topk[:, :k]


def draft_produce(target, K, seed=0, *, stream=None, out=None, out_tokens=None):
    """The synthetic draft producer on device tensors: target [B, P, V]
    (bfloat16 or float32, V contiguous), K <= P.  Returns (draft [B, K, V] of
    the target's dtype, tokens [B, K] int32); `out` may be any [B, K, V] view
    of that dtype with V contiguous."""
    lib = load()
    dev = target.device
    B, _, V = target.shape
    if out is None:
        out = torch.empty((B, K, V), dtype=target.dtype, device=dev)
    if out.dim() != 3 or tuple(out.shape) != (B, K, V) or out.dtype != target.dtype or out.stride(2) != 1:
        raise ValueError("out must be [B, K, V] of the target's dtype, contiguous along V")
    if out_tokens is None:
        out_tokens = torch.empty((B, K), dtype=torch.int32, device=dev)
    if out_tokens.dtype != torch.int32 or not out_tokens.is_contiguous() or tuple(out_tokens.shape) != (B, K):
        raise ValueError("out_tokens must be contiguous int32 [B, K]")
    td = _desc(target, "target")
    _check(lib, lib.spec_draft_produce(ctypes.byref(td), ctypes.c_int32(K), ctypes.c_uint64(seed & (2**64 - 1)),
                                       ctypes.c_void_p(out.data_ptr()), out.stride(0), out.stride(1),
                                       ctypes.c_void_p(out_tokens.data_ptr()), _stream_handle(stream, dev)))
    return out, out_tokens


def hispec_verify(final, inter, draft, draft_tokens, draft_len=None, temperature=1.0, top_p=1.0, seed=0, *,
                  stream=None, out_tokens=None, out_n_accepted=None, out_n_stage1=None):
    """The two-stage verify on device tensors: final [B, K+2, V], inter
    [B, K+1, V], draft [B, K, V] logits (same dtype, V contiguous).  Returns
    (tokens [B, K+2] int32, n_accepted [B] int32, n_stage1 [B] int32)."""
    lib = load()
    if draft_tokens.dtype != torch.int32 or not draft_tokens.is_contiguous():
        raise ValueError("draft_tokens must be contiguous int32")
    if draft_len is not None and (draft_len.dtype != torch.int32 or not draft_len.is_contiguous()):
        raise ValueError("draft_len must be contiguous int32")
    dev = final.device
    B, K2 = final.shape[0], final.shape[1]
    if out_tokens is None:
        out_tokens = torch.empty((B, K2), dtype=torch.int32, device=dev)
    if out_n_accepted is None:
        out_n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_n_stage1 is None:
        out_n_stage1 = torch.empty((B,), dtype=torch.int32, device=dev)
    fd, idd, dd = _desc(final, "final"), _desc(inter, "inter"), _desc(draft, "draft")
    _check(lib, lib.spec_hispec_verify(
        ctypes.byref(fd), ctypes.byref(idd), ctypes.byref(dd), ctypes.c_void_p(draft_tokens.data_ptr()),
        ctypes.c_void_p(draft_len.data_ptr() if draft_len is not None else None), ctypes.c_float(temperature),
        ctypes.c_float(top_p), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)), ctypes.c_void_p(out_tokens.data_ptr()),
        ctypes.c_void_p(out_n_accepted.data_ptr()), ctypes.c_void_p(out_n_stage1.data_ptr()),
        _stream_handle(stream, dev)))
    return out_tokens, out_n_accepted, out_n_stage1


def smc_step(target, draft, draft_tokens, logw_in, temperature=1.0, ess_fraction=0.5, seed=0, *, stream=None,
             out_bonus=None, out_logw=None, out_ancestor=None):
    """One SMC-SD reweight-and-resample step on device tensors.

    target [N, K+1, V], draft [N, K, V]: bfloat16 or float32, V contiguous;
    draft_tokens [N, K] int32 contiguous; logw_in [N] float64 contiguous.
    Returns (bonus [N] int32, logw [N] float64, ancestor [N] int32,
    ess [1] float64, resampled [1] int32), all on the device.
    """
    lib = load()
    if draft_tokens.dtype != torch.int32 or not draft_tokens.is_contiguous():
        raise ValueError("draft_tokens must be contiguous int32")
    if logw_in.dtype != torch.float64 or not logw_in.is_contiguous():
        raise ValueError("logw_in must be contiguous float64")
    dev = target.device
    N = target.shape[0]
    if out_bonus is None:
        out_bonus = torch.empty((N,), dtype=torch.int32, device=dev)
    if out_logw is None:
        out_logw = torch.empty((N,), dtype=torch.float64, device=dev)
    if out_ancestor is None:
        out_ancestor = torch.empty((N,), dtype=torch.int32, device=dev)
    ess = torch.empty((1,), dtype=torch.float64, device=dev)
    resampled = torch.empty((1,), dtype=torch.int32, device=dev)
    td, dd = _desc(target, "target"), _desc(draft, "draft")
    _check(lib, lib.spec_smc_step(ctypes.byref(td), ctypes.byref(dd), ctypes.c_void_p(draft_tokens.data_ptr()),
                                  ctypes.c_void_p(logw_in.data_ptr()), ctypes.c_float(temperature),
                                  ctypes.c_double(ess_fraction), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                                  ctypes.c_void_p(out_bonus.data_ptr()), ctypes.c_void_p(out_logw.data_ptr()),
                                  ctypes.c_void_p(out_ancestor.data_ptr()), ctypes.c_void_p(ess.data_ptr()),
                                  ctypes.c_void_p(resampled.data_ptr()), _stream_handle(stream, dev)))
    return out_bonus, out_logw, out_ancestor, ess, resampled


# ---- the tree round: attention of a drafted tree over a paged cache, its
# verification from given random numbers, and the cache's commit and fork.

_DTYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}
_I32, _F32 = torch.int32, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

# The argument blocks, packed in one go (an attribute of a ctypes structure
# costs about 0.15 us, and a small call launches in a few): the fields of
# SvLogits, SvTreeAttention and SvCache in order, padding where they have it.
_PACK_LOGITS = struct.Struct("@Piiiiqq").pack
_PACK_ATTENTION = struct.Struct("@iiiiiiP3qPP3q3qPP3q3qiii4xPqPPPfii4xP3qPq").pack
_PACK_CACHE = struct.Struct("@PPiiiiii4q4qPqPii").pack
_PACK_STRIDES = struct.Struct("@4q").pack
_workspaces = {}  # bytes a call needs, by its sizes; at most _KEPT of them
_KEPT = 1024
_calls = None


def _tree_calls():
    """The entry points, taking packed argument blocks."""
    global _calls
    if _calls is None:
        lib = load()
        vp, blob, i32, i64 = ctypes.c_void_p, ctypes.c_char_p, ctypes.c_int32, ctypes.c_int64

        def entry(name, args, res=ctypes.c_int):
            f = lib[name]
            f.argtypes, f.restype = args, res
            return f

        _calls = (lib, entry("spec_tree_attention", [blob, vp]), entry("spec_tree_attention_workspace", [blob], i64),
                  entry("spec_verify_tree", [blob, blob] + [vp] * 9 + [i64, vp]),
                  entry("spec_cache_commit", [blob, vp, vp, blob, blob, i32, vp, vp, vp, i64, vp, vp, vp, i64, vp]),
                  entry("spec_cache_fork", [blob, vp, vp, i64, vp, vp, vp, i64, vp]))
    return _calls


@contextlib.contextmanager
def _on(index, stream):
    """The tensors' device current, and `stream` (None: the device's current
    one), so that what is allocated meanwhile belongs to it."""
    with torch.cuda.device(index):
        if stream is None:
            yield
        else:
            if stream.device.index != index:
                raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
            with torch.cuda.stream(stream):
                yield


def _elsewhere(index, stream):
    """Whether the call has to change the current device or stream first."""
    if index < 0:
        raise ValueError("tensors must be on a GPU")
    return stream is not None or index != torch.cuda.current_device()


def _refuse(t, name, shape, dtype, index):
    kind = str(dtype).split(".")[-1]
    raise ValueError(f"{name} must be a contiguous {kind} {list(shape)} on device {index}, not {t.dtype} "
                     f"{list(t.shape)} on device {t.get_device()} with strides {list(t.stride())}")


def _array(t, name, shape, index, dtype=_I32):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, shape, dtype, index)
    return t.data_ptr()


def _rows(t, name, shape, dtype, index):
    """Checks a tensor of rows: the last axis contiguous, the others strided.
    (The library passes over the strides of axes of one.)"""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(t, name, shape, dtype, index)
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return st


def _table(t, name, B, index, width=None):
    if t.dtype is not _I32 or t.dim() != 2 or t.shape[0] != B or t.get_device() != index or \
            (width is not None and t.shape[1] != width):
        _refuse(t, name, (B, "width" if width is None else width), _I32, index)
    st, n = t.stride(), t.shape[1]
    if n > 1 and st[1] != 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    # a single row's stride may be anything
    return t.data_ptr(), (n or 1) if B == 1 else st[0]


def _workspace_bytes(lib, key, ask):
    """What `ask()` says a call with the sizes `key` needs, asked once."""
    need = _workspaces.get(key)
    if need is None:
        need = ask()
        _check(lib, need)
        if len(_workspaces) >= _KEPT:
            _workspaces.clear()
        _workspaces[key] = need
    return need


def _no_grad(*tensors):
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        raise ValueError("no backward pass: call it under torch.no_grad()")


def tree_attention(q, k_cache, v_cache, block_table, seq_len, k_tree, v_tree, parent, n_nodes=None, *, scale=None,
                   window=0, sinks=0, out=None, stream=None):
    """Attention of a drafted tree's nodes over a paged cache and their
    ancestors (spec_tree_attention).

    q [B, N, heads, dim], k_tree and v_tree [B, N, kv_heads, dim]: bfloat16 or
    float16, last axis contiguous, other strides any multiples of 8 elements.
    k_cache and v_cache [pages, page_size, kv_heads, dim] of the same dtype,
    strides likewise (a cache stored with the heads before the page's rows is
    passed transposed).  block_table [B, width], seq_len [B], parent [B, N] and
    n_nodes [B] (None: N nodes each): int32.  scale None: dim ** -0.5.  window
    0: none; sinks: the first cache rows that stay visible under a window.
    Returns out [B, N, heads, dim]; absent nodes' rows are zero.
    """
    lib, call, size_of = _tree_calls()[:3]
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [B, N, heads, dim] and k_cache [pages, page_size, kv_heads, dim]")
    dt, index = q.dtype, q.get_device()
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError(f"q: dtype {dt} is not bfloat16 or float16")
    _no_grad(q, k_cache, v_cache, k_tree, v_tree)
    shape, kc_shape = q.shape, k_cache.shape
    B, N, heads, dim = shape
    pages, page_size, kv_heads, _ = kc_shape
    t_shape = (B, N, kv_heads, dim)
    qs = _rows(q, "q", shape, dt, index)
    kts = _rows(k_tree, "k_tree", t_shape, dt, index)
    vts = _rows(v_tree, "v_tree", t_shape, dt, index)
    kcs = _rows(k_cache, "k_cache", (pages, page_size, kv_heads, dim), dt, index)
    vcs = _rows(v_cache, "v_cache", kc_shape, dt, index)
    tab, tab_stride = _table(block_table, "block_table", B, index)
    width = block_table.shape[1]
    ln = _array(seq_len, "seq_len", (B,), index)
    par = _array(parent, "parent", (B, N), index)
    nn = 0 if n_nodes is None else _array(n_nodes, "n_nodes", (B,), index)
    if out is not None:
        _rows(out, "out", shape, dt, index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return tree_attention(q, k_cache, v_cache, block_table, seq_len, k_tree, v_tree, parent, n_nodes,
                                  scale=scale, window=window, sinks=sinks, out=out)
    if out is None:
        out = q.new_empty(shape)
    os = out.stride()

    def block(ws, need):
        return _PACK_ATTENTION(_DTYPES[dt], B, N, heads, kv_heads, dim, q.data_ptr(), qs[0], qs[1], qs[2],
                               k_tree.data_ptr(), v_tree.data_ptr(), kts[0], kts[1], kts[2], vts[0], vts[1], vts[2],
                               k_cache.data_ptr(), v_cache.data_ptr(), kcs[0], kcs[1], kcs[2], vcs[0], vcs[1], vcs[2],
                               pages, page_size, width, tab, tab_stride, ln, par, nn,
                               dim ** -0.5 if scale is None else scale, window, sinks,
                               out.data_ptr(), os[0], os[1], os[2], ws, need)

    need = _workspace_bytes(lib, (index, B, N, heads, kv_heads, dim, page_size, width), lambda: size_of(block(0, 0)))
    ws = torch.empty((need,), dtype=torch.uint8, device=q.device) if need else None
    _check(lib, call(block(ws.data_ptr() if need else 0, need), _raw_stream(index)))
    return out


def _probs(t, name):
    if t.dim() != 3 or t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be [B, P, V], contiguous along V")
    if t.dtype is not _F32 and t.dtype is not torch.bfloat16:
        raise ValueError(f"{name}: dtype {t.dtype} is not float32 or bfloat16")
    (B, P, V), st = t.shape, t.stride()
    return _PACK_LOGITS(t.data_ptr(), _DTYPES[t.dtype], B, P, V, st[0], st[1])


def verify_tree(target_probs, draft_probs, tokens, parent, u_accept, u_final, n_nodes=None, *, out_tokens=None,
                out_nodes=None, out_n_accepted=None, stream=None):
    """Verification of a tree of drafted tokens against the target's
    probabilities from given random numbers (spec_verify_tree).

    target_probs [B, N, V], draft_probs [B, P, V] or None (children chosen, not
    drawn): float32 or bfloat16, V contiguous.  tokens and parent [B, N],
    n_nodes [B] (None: N nodes each): int32.  u_accept [B, N] and u_final [B]:
    float32 in [0, 1).  Returns (tokens [B, N], nodes [B, N], n_accepted [B]),
    int32.
    """
    lib, _, _, call = _tree_calls()[:4]
    td = _probs(target_probs, "target_probs")
    index = target_probs.get_device()
    dd = None
    if draft_probs is not None:
        dd = _probs(draft_probs, "draft_probs")
        if draft_probs.get_device() != index:
            raise ValueError(f"draft_probs is on {draft_probs.device}, not on {target_probs.device}")
    B, N, V = target_probs.shape
    tok = _array(tokens, "tokens", (B, N), index)
    par = _array(parent, "parent", (B, N), index)
    nn = None if n_nodes is None else _array(n_nodes, "n_nodes", (B,), index)
    ua = _array(u_accept, "u_accept", (B, N), index, _F32)
    uf = _array(u_final, "u_final", (B,), index, _F32)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return verify_tree(target_probs, draft_probs, tokens, parent, u_accept, u_final, n_nodes,
                               out_tokens=out_tokens, out_nodes=out_nodes, out_n_accepted=out_n_accepted)
    if out_tokens is None:
        out_tokens = tokens.new_empty((B, N))
    if out_nodes is None:
        out_nodes = tokens.new_empty((B, N))
    if out_n_accepted is None:
        out_n_accepted = tokens.new_empty((B,))
    need = _workspace_bytes(lib, ("verify", index, B, N, V, target_probs.dtype, dd is None),
                            lambda: lib.spec_verify_tree_workspace(B, N, V, _DTYPES[target_probs.dtype], dd is not None))
    ws = torch.empty((need,), dtype=torch.uint8, device=target_probs.device) if need else None
    _check(lib, call(td, dd, tok, par, nn, ua, uf, _array(out_tokens, "out_tokens", (B, N), index),
                     _array(out_nodes, "out_nodes", (B, N), index),
                     _array(out_n_accepted, "out_n_accepted", (B,), index), ws.data_ptr() if need else None, need,
                     _raw_stream(index)))
    return out_tokens, out_nodes, out_n_accepted


def _cache(k_cache, v_cache, block_table, seq_len, index):
    """The packed cache, its batch size and width, its shape."""
    if k_cache.dim() != 5 or seq_len.dim() != 1:
        raise ValueError("k_cache must be [layers, pages, page_size, heads, dim] and seq_len [B]")
    dt, shape = k_cache.dtype, k_cache.shape
    if dt not in _DTYPES:
        raise ValueError(f"k_cache: dtype {dt} is not float32, bfloat16 or float16")
    _no_grad(k_cache, v_cache)
    B = seq_len.shape[0]
    ks = _rows(k_cache, "k_cache", shape, dt, index)
    vs = _rows(v_cache, "v_cache", shape, dt, index)
    tab, tab_stride = _table(block_table, "block_table", B, index)
    width = block_table.shape[1]
    blob = _PACK_CACHE(k_cache.data_ptr(), v_cache.data_ptr(), _DTYPES[dt], *shape, ks[0], ks[1], ks[2], ks[3], vs[0],
                       vs[1], vs[2], vs[3], tab, tab_stride, _array(seq_len, "seq_len", (B,), index), B, width)
    return blob, B, width, shape


def _cache_outs(seq_len, B, width, index, out_table, out_len, out_status):
    if out_table is None:
        out_table = seq_len.new_empty((B, width))
    if out_len is None:
        out_len = seq_len.new_empty((B,))
    if out_status is None:
        out_status = seq_len.new_empty((1,))
    tab, stride = _table(out_table, "out_table", B, index, width)
    return (out_table, out_len, out_status), (tab, stride, _array(out_len, "out_len", (B,), index),
                                              _array(out_status, "out_status", (1,), index))


def _cache_workspace(lib, like, B, N, page_size):
    need = _workspace_bytes(lib, (B, N, page_size), lambda: lib.spec_cache_workspace(B, N, page_size))
    return torch.empty((need,), dtype=torch.uint8, device=like.device), need


def cache_commit(k_cache, v_cache, block_table, seq_len, k_tree, v_tree, nodes, n_accepted, *, out_table=None,
                 out_len=None, out_status=None, stream=None):
    """Append every sequence's accepted path to the cache (spec_cache_commit).

    k_cache, v_cache [layers, pages, page_size, heads, dim] (float32, bfloat16
    or float16), written in place; k_tree, v_tree [layers, B, N, heads, dim];
    block_table [B, width], seq_len [B], nodes [B, N] (None: nodes 0..n, a
    chain) and n_accepted [B]: int32.  Returns (table, length, status): new
    tensors, or out_table and out_len, which may be block_table and seq_len
    themselves.  status [1]: 0, the number of pages lacking, or -1 for bad
    indices or a shared page that would be appended to; unless 0, nothing was
    appended.
    """
    lib, _, _, _, call, _ = _tree_calls()
    index = k_cache.get_device()
    blob, B, width, shape = _cache(k_cache, v_cache, block_table, seq_len, index)
    _no_grad(k_tree, v_tree)
    if k_tree.dim() != 5:
        raise ValueError("k_tree must be [layers, B, N, heads, dim]")
    N = k_tree.shape[2]
    want = (shape[0], B, N, shape[3], shape[4])
    kts = _rows(k_tree, "k_tree", want, k_cache.dtype, index)
    vts = _rows(v_tree, "v_tree", want, k_cache.dtype, index)
    nd = None if nodes is None else _array(nodes, "nodes", (B, N), index)
    na = _array(n_accepted, "n_accepted", (B,), index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return cache_commit(k_cache, v_cache, block_table, seq_len, k_tree, v_tree, nodes, n_accepted,
                                out_table=out_table, out_len=out_len, out_status=out_status)
    outs, ptrs = _cache_outs(seq_len, B, width, index, out_table, out_len, out_status)
    ws, need = _cache_workspace(lib, k_cache, B, N, shape[2])
    _check(lib, call(blob, k_tree.data_ptr(), v_tree.data_ptr(), _PACK_STRIDES(*kts[:4]), _PACK_STRIDES(*vts[:4]), N,
                     nd, na, *ptrs, ws.data_ptr(), need, _raw_stream(index)))
    return outs


def cache_fork(k_cache, v_cache, block_table, seq_len, ancestor, *, out_table=None, out_len=None, out_status=None,
               stream=None):
    """Continue slot k of the batch as sequence ancestor[k], -1 freeing the
    slot (spec_cache_fork): full pages are shared, partly filled last pages
    copied.  ancestor [B] int32, as smc_step returns it; the rest as
    cache_commit, with outputs apart from block_table and seq_len.
    """
    lib, _, _, _, _, call = _tree_calls()
    index = k_cache.get_device()
    blob, B, width, shape = _cache(k_cache, v_cache, block_table, seq_len, index)
    anc = _array(ancestor, "ancestor", (B,), index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return cache_fork(k_cache, v_cache, block_table, seq_len, ancestor, out_table=out_table, out_len=out_len,
                              out_status=out_status)
    outs, ptrs = _cache_outs(seq_len, B, width, index, out_table, out_len, out_status)
    ws, need = _cache_workspace(lib, k_cache, B, 0, shape[2])
    _check(lib, call(blob, anc, *ptrs, ws.data_ptr(), need, _raw_stream(index)))
    return outs


# ---- latent rows: one row per token, shared by the heads

# the fields of sv_latent_attention, sv_head_product, sv_cache_rows and sv_latent_prompt in order
_PACK_LATENT = struct.Struct("@iiiiiiP3qP2qP2qiii4xPqPPPf4xP3qPq").pack
_PACK_PRODUCT = struct.Struct("@iiiii4xP2qP2qP2q").pack
_PACK_WRITE = struct.Struct("@P2qiiiiiiPqPqP").pack
_PACK_PROMPT = struct.Struct("@iiiiiiiii4xP2qP2qiii4xPqPPP2qP2qf4xP2qPq").pack
_latent = None


def _latent_calls():
    """The entry points, taking packed argument blocks."""
    global _latent
    if _latent is None:
        lib = load()
        vp, blob, i32, i64 = ctypes.c_void_p, ctypes.c_char_p, ctypes.c_int32, ctypes.c_int64

        def entry(name, args, res=ctypes.c_int):
            f = lib[name]
            f.argtypes, f.restype = args, res
            return f

        _latent = (lib, entry("spec_latent_attention", [blob, vp]),
                   entry("spec_latent_attention_workspace", [blob], i64), entry("spec_head_product", [blob, vp]),
                   entry("spec_latent_prompt", [blob, vp]), entry("spec_latent_prompt_workspace", [blob], i64),
                   entry("spec_cache_reserve", [vp, i64, vp, vp, i32, i32, i32, i32, i32, vp, i64, vp, vp, vp, vp, vp, vp,
                                                i64, vp]),
                   entry("spec_cache_reserve_workspace", [i32, i32, i32], i64), entry("spec_cache_write", [blob, vp]),
                   entry("spec_beam_select", [blob, vp, vp, i32, vp, vp, vp, vp, vp, i64, vp]),
                   entry("spec_beam_workspace", [i32, i32, i32], i64),
                   entry("spec_beam_reorder", [vp, i64, vp, i64, i64, i32, vp, vp]))
    return _latent


def _half(t, name):
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
        raise ValueError(f"{name}: dtype {t.dtype} is not bfloat16 or float16")
    return t.dtype


def _int32(x, name):
    """An argument that ctypes would cut to 32 bits."""
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name}: {x} is out of range")
    return x


def _tokens(t, name, shape, dtype, index):
    """_rows for a tensor that may be empty (whose strides mean nothing)."""
    if shape[0] == 0 and t.dtype is dtype and t.shape == shape and t.get_device() == index:
        return (0,) * len(shape)
    return _rows(t, name, shape, dtype, index)


def latent_attention(q, cache, block_table, seq_len, rows, parent=None, n_nodes=None, *, dim_v, scale, out=None,
                     stream=None):
    """Attention of new tokens or a drafted tree's nodes on a paged cache of
    latent rows and their ancestors' rows (spec_latent_attention).

    q [B, N, heads, dim], cache [pages, page_size, dim] and the nodes' own rows
    [B, N, dim]: bfloat16 or float16, last axis contiguous, other strides any
    multiples of 8 elements.  block_table [B, width], seq_len [B], parent
    [B, N] (None: chains) and n_nodes [B] (None: N nodes each): int32.  Values
    are the rows' first dim_v elements.  Returns out [B, N, heads, dim_v];
    absent nodes' rows are zero.
    """
    lib, call, size_of = _latent_calls()[:3]
    if q.dim() != 4 or cache.dim() != 3:
        raise ValueError("q must be [B, N, heads, dim] and cache [pages, page_size, dim]")
    dt, index = _half(q, "q"), q.get_device()
    _no_grad(q, cache, rows)
    shape = q.shape
    B, N, heads, dim = shape
    pages, page_size, _ = cache.shape
    qs = _rows(q, "q", shape, dt, index)
    cs = _rows(cache, "cache", (pages, page_size, dim), dt, index)
    rs = _rows(rows, "rows", (B, N, dim), dt, index)
    tab, tab_stride = _table(block_table, "block_table", B, index)
    width = block_table.shape[1]
    ln = _array(seq_len, "seq_len", (B,), index)
    par = 0 if parent is None else _array(parent, "parent", (B, N), index)
    nn = 0 if n_nodes is None else _array(n_nodes, "n_nodes", (B,), index)
    out_shape = (B, N, heads, dim_v)
    if out is not None:
        _rows(out, "out", out_shape, dt, index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return latent_attention(q, cache, block_table, seq_len, rows, parent, n_nodes, dim_v=dim_v, scale=scale,
                                    out=out)
    if out is None:
        out = q.new_empty(out_shape)
    os = out.stride()

    def block(ws, need):
        return _PACK_LATENT(_DTYPES[dt], B, N, heads, dim, dim_v, q.data_ptr(), qs[0], qs[1], qs[2], rows.data_ptr(),
                            rs[0], rs[1], cache.data_ptr(), cs[0], cs[1], pages, page_size, width, tab, tab_stride, ln,
                            par, nn, scale, out.data_ptr(), os[0], os[1], os[2], ws, need)

    need = _workspace_bytes(lib, ("latent", index, B, N, heads, dim, dim_v, page_size, width),
                            lambda: size_of(block(0, 0)))
    ws = torch.empty((need,), dtype=torch.uint8, device=q.device) if need else None
    _check(lib, call(block(ws.data_ptr() if need else 0, need), _raw_stream(index)))
    return out


def head_product(x, w, *, out=None, stream=None):
    """out[t, h] = w[h] x[t, h] (spec_head_product): queries into the latent
    space, results out of it.

    x [T, heads, K], w [heads, M, K]: bfloat16 or float16, last axis contiguous,
    other strides any multiples of 8 elements.  Returns out [T, heads, M].
    """
    lib, _, _, call = _latent_calls()[:4]
    if x.dim() != 3 or w.dim() != 3:
        raise ValueError("x must be [T, heads, K] and w [heads, M, K]")
    dt, index = _half(x, "x"), x.get_device()
    _no_grad(x, w)
    (T, heads, K), M = x.shape, w.shape[1]
    xs = _tokens(x, "x", x.shape, dt, index)
    ws = _rows(w, "w", (heads, M, K), dt, index)
    if out is not None:
        _tokens(out, "out", (T, heads, M), dt, index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return head_product(x, w, out=out)
    if out is None:
        out = x.new_empty((T, heads, M))
    os = out.stride()
    _check(lib, call(_PACK_PRODUCT(_DTYPES[dt], T, heads, K, M, x.data_ptr(), xs[0], xs[1], w.data_ptr(), ws[0], ws[1],
                                   out.data_ptr(), os[0], os[1]), _raw_stream(index)))
    return out


def latent_prompt(q, cache, block_table, seq_len, q_start, w_k, w_v, *, rows, scale=None, out=None, stream=None):
    """Causal attention of prompts over a paged cache of latent rows, with keys
    and values expanded per head (spec_latent_prompt).

    q [T, heads, dim_k + dim_p]: rows q_start[b] .. q_start[b + 1] are the last
    tokens of sequence b, whose rows are in the cache already.  cache [pages,
    page_size, latent + dim_p], w_k [heads, dim_k, latent], w_v [heads, dim_v,
    latent]: one dtype, bfloat16 or float16, last axis contiguous, other strides
    any multiples of 8 elements.  block_table [B, width], seq_len [B], q_start
    [B + 1]: int32.  rows: at least the sum of the lengths (it sizes the
    workspace; what does not fit comes out as NaN).  scale None: (dim_k +
    dim_p) ** -0.5.  Returns out [T, heads, dim_v]; rows of q that belong to no
    sequence are not written.
    """
    lib, _, _, _, call, size_of = _latent_calls()[:6]
    if q.dim() != 3 or cache.dim() != 3 or w_k.dim() != 3 or w_v.dim() != 3 or seq_len.dim() != 1:
        raise ValueError("q must be [T, heads, dim], cache [pages, page_size, dim], w_k and w_v [heads, dim, latent] "
                         "and seq_len [B]")
    dt, index = _half(q, "q"), q.get_device()
    _no_grad(q, cache, w_k, w_v)
    T, heads, dim = q.shape
    pages, page_size, whole = cache.shape
    dim_k, latent = w_k.shape[1:]
    dim_p, dim_v, B = whole - latent, w_v.shape[1], seq_len.shape[0]
    if dim != dim_k + dim_p:
        raise ValueError(f"q has {dim} elements a head; w_k and the cache make it {dim_k} + {dim_p}")
    _int32(rows, "rows")
    qs = _tokens(q, "q", q.shape, dt, index)
    cs = _rows(cache, "cache", cache.shape, dt, index)
    wks = _rows(w_k, "w_k", (heads, dim_k, latent), dt, index)
    wvs = _rows(w_v, "w_v", (heads, dim_v, latent), dt, index)
    tab, tab_stride = _table(block_table, "block_table", B, index)
    width = block_table.shape[1]
    ln = _array(seq_len, "seq_len", (B,), index)
    start = _array(q_start, "q_start", (B + 1,), index)
    if out is not None:
        _tokens(out, "out", (T, heads, dim_v), dt, index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return latent_prompt(q, cache, block_table, seq_len, q_start, w_k, w_v, rows=rows, scale=scale, out=out)
    if out is None:
        out = q.new_empty((T, heads, dim_v))
    os = out.stride()

    def block(ws, need):
        return _PACK_PROMPT(_DTYPES[dt], T, B, heads, latent, dim_k, dim_p, dim_v, rows, q.data_ptr(), qs[0], qs[1],
                            cache.data_ptr(), cs[0], cs[1], pages, page_size, width, tab, tab_stride, ln, start,
                            w_k.data_ptr(), wks[0], wks[1], w_v.data_ptr(), wvs[0], wvs[1],
                            dim ** -0.5 if scale is None else scale, out.data_ptr(), os[0], os[1], ws, need)

    need = _workspace_bytes(lib, ("prompt", B, T, heads, latent, dim_k, dim_p, dim_v, rows, page_size, width),
                            lambda: size_of(block(0, 0)))
    ws = torch.empty((need,), dtype=torch.uint8, device=q.device)
    _check(lib, call(block(ws.data_ptr(), need), _raw_stream(index)))
    return out


def cache_reserve(block_table, seq_len, n_new, *, pages, page_size, rows, out_table=None, out_len=None, stream=None):
    """Room for n_new[b] more rows of every sequence, and where they go
    (spec_cache_reserve).

    block_table [B, width], seq_len [B], n_new [B]: int32.  pages and page_size:
    the cache's.  rows: at least the sum of n_new, the length of the lists.
    Returns (table, length, start [B + 1], slots [rows], position [rows], status
    [1]), int32; out_table and out_len may be block_table and seq_len themselves.
    status: 0, the number of pages lacking, or -1; unless 0, nothing is reserved.
    """
    lib, call, size_of = _latent_calls()[0], _latent_calls()[6], _latent_calls()[7]
    index = seq_len.get_device()
    if seq_len.dim() != 1:
        raise ValueError("seq_len must be [B]")
    for x, name in ((pages, "pages"), (page_size, "page_size"), (rows, "rows")):
        _int32(x, name)
    B = seq_len.shape[0]
    tab, tab_stride = _table(block_table, "block_table", B, index)
    width = block_table.shape[1]
    ln, nn = _array(seq_len, "seq_len", (B,), index), _array(n_new, "n_new", (B,), index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return cache_reserve(block_table, seq_len, n_new, pages=pages, page_size=page_size, rows=rows,
                                 out_table=out_table, out_len=out_len)
    if out_table is None:
        out_table = seq_len.new_empty((B, width))
    if out_len is None:
        out_len = seq_len.new_empty((B,))
    new, stride = _table(out_table, "out_table", B, index, width)
    new_len = _array(out_len, "out_len", (B,), index)
    need = _workspace_bytes(lib, ("reserve", B, page_size, rows), lambda: size_of(B, page_size, rows))
    # one allocation: the lists and starts, the status and the workspace
    both = seq_len.new_empty((2 * rows + B + 2 + need // 4,))
    slots, position, start, status, ws = torch.split(both, (rows, rows, B + 1, 1, need // 4))
    _check(lib, call(tab, tab_stride, ln, nn, B, width, pages, page_size, rows, new, stride, new_len, start.data_ptr(),
                     slots.data_ptr(), position.data_ptr(), status.data_ptr(), ws.data_ptr(), need, _raw_stream(index)))
    return out_table, out_len, start, slots, position, status


def cache_write(cache, slots, a, b=None, *, stream=None):
    """Rows into their slots of a paged cache (spec_cache_write): row t of a, and
    of b behind it, into slot slots[t], -1 for none.

    cache [pages, page_size, dim] (float32, bfloat16 or float16), written in
    place; a [T, dim_a] and b [T, dim_b] (None: nothing) of the same dtype with
    dim_a + dim_b = dim; last axes contiguous, other strides any multiples of 16
    bytes.  slots [T] int32, no slot twice.
    """
    lib, call = _latent_calls()[0], _latent_calls()[8]
    if cache.dim() != 3 or a.dim() != 2:
        raise ValueError("cache must be [pages, page_size, dim] and a [T, dim_a]")
    dt, index = cache.dtype, cache.get_device()
    if dt not in _DTYPES:
        raise ValueError(f"cache: dtype {dt} is not float32, bfloat16 or float16")
    _no_grad(cache, a) if b is None else _no_grad(cache, a, b)
    pages, page_size, dim = cache.shape
    T, dim_a = a.shape
    dim_b = dim - dim_a
    cs = _rows(cache, "cache", cache.shape, dt, index)
    st_a = _tokens(a, "a", a.shape, dt, index)
    if b is None:
        if dim_b:
            raise ValueError(f"rows of {dim_a} elements for a cache of {dim}")
        at_b, st_b = 0, (0,)
    else:
        st_b = _tokens(b, "b", (T, dim_b), dt, index)
        at_b = b.data_ptr()
    where = _array(slots, "slots", (T,), index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return cache_write(cache, slots, a, b)
    _check(lib, call(_PACK_WRITE(cache.data_ptr(), cs[0], cs[1], _DTYPES[dt], pages, page_size, T, dim_a, dim_b,
                                 a.data_ptr(), st_a[0], at_b, st_b[0], where), _raw_stream(index)))


def beam_select(logits, scores, finished=None, *, end=-1, out_tokens=None, out_ancestor=None, out_scores=None,
                out_finished=None, stream=None):
    """The W best continuations of every sequence's W beams (spec_beam_select).

    logits [B, W, V]: float32 or bfloat16, V contiguous.  scores [B, W] float32,
    the beams' running log-probabilities (-inf: no such beam).  finished [B, W]
    int32 or None; end: the token that finishes a beam, -1 for none.  Returns
    (tokens [B, W] int32, ancestor [B * W] int32, as cache_fork and beam_reorder
    take it, scores [B, W] float32, finished [B, W] int32), best first.
    """
    lib, call, size_of = _latent_calls()[0], _latent_calls()[9], _latent_calls()[10]
    desc = _probs(logits, "logits")
    index = logits.get_device()
    B, W, V = logits.shape
    _int32(end, "end")
    _no_grad(logits, scores)
    sc = _array(scores, "scores", (B, W), index, _F32)
    fin = None if finished is None else _array(finished, "finished", (B, W), index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return beam_select(logits, scores, finished, end=end, out_tokens=out_tokens, out_ancestor=out_ancestor,
                               out_scores=out_scores, out_finished=out_finished)
    if out_tokens is None:
        out_tokens = torch.empty((B, W), dtype=_I32, device=logits.device)
    if out_ancestor is None:
        out_ancestor = torch.empty((B * W,), dtype=_I32, device=logits.device)
    if out_scores is None:
        out_scores = scores.new_empty((B, W))
    if out_finished is None:
        out_finished = torch.empty((B, W), dtype=_I32, device=logits.device)
    need = _workspace_bytes(lib, ("beam", index, B, W, V), lambda: size_of(B, W, V))
    ws = torch.empty((need,), dtype=torch.uint8, device=logits.device)
    _check(lib, call(desc, sc, fin, end, _array(out_tokens, "out_tokens", (B, W), index),
                     _array(out_ancestor, "out_ancestor", (B * W,), index),
                     _array(out_scores, "out_scores", (B, W), index, _F32),
                     _array(out_finished, "out_finished", (B, W), index), ws.data_ptr(), need, _raw_stream(index)))
    return out_tokens, out_ancestor, out_scores, out_finished


def beam_reorder(state, ancestor, *, out=None, stream=None):
    """Rows of a state in the order of their ancestors (spec_beam_reorder): row k
    of the result is row ancestor[k] of state, any dtype, [rows, ...], rows
    contiguous in themselves.  Where ancestor[k] is -1, row k of out is zero.
    """
    lib, call = _latent_calls()[0], _latent_calls()[11]
    index = state.get_device()
    _no_grad(state)
    if state.dim() < 1:
        raise ValueError("state must be [rows, ...]")
    for t in (state,) if out is None else (state, out):
        if t.is_conj() or t.is_neg():
            raise ValueError("lazily conjugated or negated: resolve it first")
    n = state.shape[0]
    anc = _array(ancestor, "ancestor", (n,), index)
    if _elsewhere(index, stream):
        with _on(index, stream):
            return beam_reorder(state, ancestor, out=out)
    if out is None:
        out = torch.empty(state.shape, dtype=state.dtype, device=state.device)
    elif out.shape != state.shape or out.dtype is not state.dtype or out.get_device() != index:
        raise ValueError(f"out must be {state.dtype} {list(state.shape)} on device {index}")
    if n == 0:
        return out
    if not (state.is_contiguous() or state[0].is_contiguous()) or not (out.is_contiguous() or out[0].is_contiguous()):
        raise ValueError("rows must be contiguous")
    size = state.element_size()
    _check(lib, call(state.data_ptr(), state.stride(0) * size, out.data_ptr(), out.stride(0) * size,
                     state.numel() // n * size, n, anc, _raw_stream(index)))
    return out


def profile_enable(on=True):
    load().spec_verify_profile_enable(1 if on else 0)


def profile_read():
    """{kind: (summed ms, launches)} since the previous read (synchronises)."""
    lib = load()
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    rc = lib.spec_verify_profile_read(ms, cnt, n)
    _check(lib, rc)
    return {KERNEL_KINDS[i]: (ms[i], cnt[i]) for i in range(n)}


def release():
    load().spec_verify_release()


def stream_read(buf, sink, unroll=4, stream=None):
    """Launch the streaming-read calibration kernel over a device tensor."""
    lib = load()
    sh = _stream_handle(stream, buf.device)
    _check(lib, lib.spec_verify_stream_read(ctypes.c_void_p(buf.data_ptr()), buf.numel() * buf.element_size(),
                                            ctypes.c_void_p(sink.data_ptr()), unroll, sh))
