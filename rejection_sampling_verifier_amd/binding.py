"""ctypes binding of libspecverify.so.

Argument marshalling only: every step of the verify computation runs in the
library's HIP kernels.  PyTorch provides device memory and the current
stream.  There is no fallback: when the library is missing or no GPU is
present, the calls raise.
"""

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_F32, SV_BF16, SV_F16 = 0, 1, 2
MAX_NODES = 64
PROBE_POS, PROBE_ROW = 8, 4
STATUS = {0: "SV_OK", -1: "SV_EINVAL", -2: "SV_ESHAPE", -3: "SV_EDTYPE", -4: "SV_EHIP", -5: "SV_ENOMEM",
          -6: "SV_EALIGN", -7: "SV_ECAPTURE", -8: "SV_ETOOBIG"}
KERNEL_KINDS = ("stats", "topp", "rows", "smc", "produce", "tree_attention", "tree_join", "tree_verify", "cache_plan",
                "cache_copy")

EXPORTS = ("spec_verify", "spec_verify_noalloc", "spec_verify_probe", "spec_greedy_verify", "spec_hispec_verify", "spec_smc_step",
           "spec_draft_produce",
           "spec_tree_attention", "spec_tree_attention_workspace", "spec_verify_tree",
           "spec_cache_commit", "spec_cache_fork", "spec_cache_workspace",
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
    lib.spec_verify_tree.argtypes = [P(SvLogits), P(SvLogits)] + [vp] * 9
    lib.spec_verify_tree.restype = ctypes.c_int
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
_I64x3, _I64x4 = ctypes.c_int64 * 3, ctypes.c_int64 * 4


@contextlib.contextmanager
def _launch(dev, stream):
    """The stream to launch on, its device current and the stream current, so
    that what is allocated meanwhile belongs to it."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {dev}")
    if stream is None and (dev.index is None or dev.index == torch.cuda.current_device()):
        yield torch.cuda.current_stream(dev).cuda_stream
        return
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream(dev).cuda_stream
        else:
            if stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _ints(t, name, shape, dev, dtype=torch.int32):
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {str(dtype).split('.')[-1]} {list(shape)}, not {t.dtype} "
                         f"{list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    return t.data_ptr()


def _table(t, name, B, dev, width=None):
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != B or (t.shape[1] > 1 and t.stride(1) != 1) or \
            (width is not None and t.shape[1] != width):
        raise ValueError(f"{name} must be int32 [{B}, {'width' if width is None else width}], contiguous along its rows")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    # a single row's stride may be anything
    return t.data_ptr(), max(t.shape[1], 1) if B == 1 else t.stride(0)


def _rows(t, name, shape, like):
    """Pointer and strides of a tensor of rows; the stride of an axis of one is
    of no meaning and may be anything."""
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype != like.dtype:
        raise ValueError(f"{name} is {t.dtype}, not {like.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return t.data_ptr(), [0 if n == 1 else s for n, s in zip(t.shape[:-1], t.stride()[:-1])]


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
    lib = load()
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [B, N, heads, dim] and k_cache [pages, page_size, kv_heads, dim]")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"q: dtype {q.dtype} is not bfloat16 or float16")
    _no_grad(q, k_cache, v_cache, k_tree, v_tree)
    dev = q.device
    B, N, heads, dim = q.shape
    pages, page_size, kv_heads, _ = k_cache.shape
    a = SvTreeAttention()
    a.dtype, a.B, a.N, a.heads, a.kv_heads, a.dim = _DTYPES[q.dtype], B, N, heads, kv_heads, dim
    a.pages, a.page_size = pages, page_size
    a.q, st = _rows(q, "q", (B, N, heads, dim), q)
    a.q_stride = _I64x3(*st)
    a.k_tree, st = _rows(k_tree, "k_tree", (B, N, kv_heads, dim), q)
    a.k_tree_stride = _I64x3(*st)
    a.v_tree, st = _rows(v_tree, "v_tree", (B, N, kv_heads, dim), q)
    a.v_tree_stride = _I64x3(*st)
    a.k_cache, st = _rows(k_cache, "k_cache", (pages, page_size, kv_heads, dim), q)
    a.k_cache_stride = _I64x3(*st)
    a.v_cache, st = _rows(v_cache, "v_cache", (pages, page_size, kv_heads, dim), q)
    a.v_cache_stride = _I64x3(*st)
    a.table, a.table_stride = _table(block_table, "block_table", B, dev)
    a.width = block_table.shape[1]
    a.len = _ints(seq_len, "seq_len", (B,), dev)
    a.parent = _ints(parent, "parent", (B, N), dev)
    a.n_nodes = None if n_nodes is None else _ints(n_nodes, "n_nodes", (B,), dev)
    a.scale = dim ** -0.5 if scale is None else scale
    a.window, a.sinks = window, sinks
    with _launch(dev, stream) as sh:
        if out is None:
            out = torch.empty((B, N, heads, dim), dtype=q.dtype, device=dev)
        a.out, st = _rows(out, "out", (B, N, heads, dim), q)
        a.out_stride = _I64x3(*st)
        need = lib.spec_tree_attention_workspace(a)
        _check(lib, need)
        if need:
            ws = torch.empty((need,), dtype=torch.uint8, device=dev)
            a.workspace, a.workspace_bytes = ws.data_ptr(), need
        _check(lib, lib.spec_tree_attention(a, sh))
    return out


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
    lib = load()
    dev = target_probs.device
    td = _desc(target_probs, "target_probs")
    dd = None
    if draft_probs is not None:
        dd = _desc(draft_probs, "draft_probs")
        if draft_probs.device != dev:
            raise ValueError(f"draft_probs is on {draft_probs.device}, not on {dev}")
    B, N, _ = target_probs.shape
    ins = (_ints(tokens, "tokens", (B, N), dev), _ints(parent, "parent", (B, N), dev),
           None if n_nodes is None else _ints(n_nodes, "n_nodes", (B,), dev),
           _ints(u_accept, "u_accept", (B, N), dev, torch.float32), _ints(u_final, "u_final", (B,), dev, torch.float32))
    with _launch(dev, stream) as sh:
        if out_tokens is None:
            out_tokens = torch.empty((B, N), dtype=torch.int32, device=dev)
        if out_nodes is None:
            out_nodes = torch.empty((B, N), dtype=torch.int32, device=dev)
        if out_n_accepted is None:
            out_n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        _check(lib, lib.spec_verify_tree(td, dd, *ins, _ints(out_tokens, "out_tokens", (B, N), dev),
                                         _ints(out_nodes, "out_nodes", (B, N), dev),
                                         _ints(out_n_accepted, "out_n_accepted", (B,), dev), sh))
    return out_tokens, out_nodes, out_n_accepted


def _cache(k_cache, v_cache, block_table, seq_len):
    if k_cache.dim() != 5:
        raise ValueError("k_cache must be [layers, pages, page_size, heads, dim]")
    if k_cache.dtype not in _DTYPES:
        raise ValueError(f"k_cache: dtype {k_cache.dtype} is not float32, bfloat16 or float16")
    _no_grad(k_cache, v_cache)
    dev, shape = k_cache.device, tuple(k_cache.shape)
    B = seq_len.shape[0]
    c = SvCache()
    c.dtype = _DTYPES[k_cache.dtype]
    c.layers, c.pages, c.page_size, c.heads, c.dim = shape
    c.k, st = _rows(k_cache, "k_cache", shape, k_cache)
    c.k_stride = _I64x4(*st)
    c.v, st = _rows(v_cache, "v_cache", shape, k_cache)
    c.v_stride = _I64x4(*st)
    c.table, c.table_stride = _table(block_table, "block_table", B, dev)
    c.len = _ints(seq_len, "seq_len", (B,), dev)
    c.B, c.width = B, block_table.shape[1]
    return c


def _cache_outs(c, dev, out_table, out_len, out_status):
    if out_table is None:
        out_table = torch.empty((c.B, c.width), dtype=torch.int32, device=dev)
    if out_len is None:
        out_len = torch.empty((c.B,), dtype=torch.int32, device=dev)
    if out_status is None:
        out_status = torch.empty((1,), dtype=torch.int32, device=dev)
    tab, stride = _table(out_table, "out_table", c.B, dev, c.width)
    return (out_table, out_len, out_status), (tab, stride, _ints(out_len, "out_len", (c.B,), dev),
                                              _ints(out_status, "out_status", (1,), dev))


def cache_commit(k_cache, v_cache, block_table, seq_len, k_tree, v_tree, nodes, n_accepted, *, out_table=None,
                 out_len=None, out_status=None, stream=None):
    """Append every sequence's accepted path to the cache (spec_cache_commit).

    k_cache, v_cache [layers, pages, page_size, heads, dim] (float32, bfloat16
    or float16), written in place; k_tree, v_tree [layers, B, N, heads, dim];
    block_table [B, width], seq_len [B], nodes [B, N] (None: nodes 0..n, a
    chain) and n_accepted [B]: int32.  Returns (table, length, status): new
    tensors, or out_table and out_len, which may be block_table and seq_len
    themselves.  status [1]: 0, the number of pages lacking, or -1 for bad
    indices; unless 0, nothing was appended.
    """
    lib = load()
    c = _cache(k_cache, v_cache, block_table, seq_len)
    _no_grad(k_tree, v_tree)
    dev = k_cache.device
    if k_tree.dim() != 5:
        raise ValueError("k_tree must be [layers, B, N, heads, dim]")
    N = k_tree.shape[2]
    want = (c.layers, c.B, N, c.heads, c.dim)
    kt, kst = _rows(k_tree, "k_tree", want, k_cache)
    vt, vst = _rows(v_tree, "v_tree", want, k_cache)
    nd = None if nodes is None else _ints(nodes, "nodes", (c.B, N), dev)
    na = _ints(n_accepted, "n_accepted", (c.B,), dev)
    with _launch(dev, stream) as sh:
        outs, ptrs = _cache_outs(c, dev, out_table, out_len, out_status)
        need = lib.spec_cache_workspace(c.B, N, c.page_size)
        _check(lib, need)
        ws = torch.empty((need,), dtype=torch.uint8, device=dev)
        _check(lib, lib.spec_cache_commit(c, kt, vt, _I64x4(*kst), _I64x4(*vst), N, nd, na, *ptrs, ws.data_ptr(), need,
                                          sh))
    return outs


def cache_fork(k_cache, v_cache, block_table, seq_len, ancestor, *, out_table=None, out_len=None, out_status=None,
               stream=None):
    """Continue slot k of the batch as sequence ancestor[k], -1 freeing the
    slot (spec_cache_fork): full pages are shared, partly filled last pages
    copied.  ancestor [B] int32, as smc_step returns it; the rest as
    cache_commit, with outputs apart from block_table and seq_len.
    """
    lib = load()
    c = _cache(k_cache, v_cache, block_table, seq_len)
    dev = k_cache.device
    anc = _ints(ancestor, "ancestor", (c.B,), dev)
    with _launch(dev, stream) as sh:
        outs, ptrs = _cache_outs(c, dev, out_table, out_len, out_status)
        need = lib.spec_cache_workspace(c.B, 0, c.page_size)
        _check(lib, need)
        ws = torch.empty((need,), dtype=torch.uint8, device=dev)
        _check(lib, lib.spec_cache_fork(c, anc, *ptrs, ws.data_ptr(), need, sh))
    return outs


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
