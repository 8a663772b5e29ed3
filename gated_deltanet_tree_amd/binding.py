"""ctypes binding of libgdn_tree.so -- argument marshalling only.

Every computation runs in the HIP library; this module converts numpy arrays and torch
tensors (device memory on ROCm) into the pointers and sizes that include/gdn_tree.h
declares, and raises GdnError on a non-zero status.  torch is imported before the library is
loaded so that both share one HIP runtime.  There is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdn_tree.so")

GDN_F32, GDN_BF16 = 0, 1
STATUS = {0: "GDN_OK", -1: "GDN_EINVAL", -2: "GDN_ETREE", -3: "GDN_EPATH",
          -4: "GDN_ECAPACITY", -5: "GDN_EDEVICE"}
EXPORTS = [
    "gdn_last_error", "gdn_schedule_words", "gdn_hld_schedule", "gdn_ddtree_build",
    "gdn_verify_workspace_bytes",
    "gdn_tree_verify", "gdn_tree_verify_noalloc", "gdn_tree_verify_wave",
    "gdn_tree_verify_wave_timed",
    "gdn_tree_verify_ut", "gdn_tree_verify_ut_timed", "gdn_tree_conv",
    "gdn_tree_conv_verify", "gdn_tree_conv_verify_timed",
    "gdn_commit_path", "gdn_prefill", "gdn_prefill_timed",
    "gdn_compact_factors", "gdn_flush",
    "gdn_kv_append", "gdn_kv_commit", "gdn_kv_read",
    "gdn_attention_workspace_bytes", "gdn_attention", "gdn_tree_attention",
    "gdn_kv_bounds", "gdn_kv_select", "gdn_sparse_workspace_bytes", "gdn_sparse_attention",
    "gdn_sparse_tree_attention",
    "gdn_accept_workspace_bytes", "gdn_tree_accept",
    "gdn_logprobs_workspace_bytes", "gdn_token_logprobs",
    "gdn_pages_workspace_bytes", "gdn_kv_reserve", "gdn_kv_release",
]
IMAGE_HEADER = 16
IMAGE_MAGIC = 0x53444E47


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str, text: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {text}")
        self.status = status


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I32P = ctypes.POINTER(ctypes.c_int32)
_FP = ctypes.POINTER(ctypes.c_float)


class VerifyArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _I32), ("n_heads", _I32), ("head_dim", _I32), ("n_nodes", _I32),
        ("max_nodes", _I32), ("layer_begin", _I32), ("n_layers", _I32), ("in_dtype", _I32),
        ("q", _P), ("k", _P), ("v", _P), ("beta", _P), ("gate", _P), ("state", _P),
        ("bank_k", _P * 2), ("bank_u", _P * 2), ("bank_lg", _P * 2),
        ("role", _P), ("pending_len", _P), ("pending_rows", _P), ("workspace", _P), ("out", _P),
    ]


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _I32), ("n_heads", _I32), ("head_dim", _I32), ("n_tokens", _I32),
        ("layer_begin", _I32), ("n_layers", _I32), ("in_dtype", _I32), ("reserved", _I32),
        ("q", _P), ("k", _P), ("v", _P), ("beta", _P), ("gate", _P), ("seq_offsets", _P),
        ("state", _P), ("out", _P),
    ]


class ConvArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _I32), ("channels", _I32), ("width", _I32), ("n_nodes", _I32),
        ("max_nodes", _I32), ("layer_begin", _I32), ("n_layers", _I32), ("in_dtype", _I32),
        ("x", _P), ("weight", _P), ("conv_state", _P), ("bank_x", _P * 2),
        ("role", _P), ("pending_len", _P), ("pending_rows", _P), ("out", _P),
    ]


class KvArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _I32), ("n_heads", _I32), ("n_kv_heads", _I32), ("head_dim", _I32),
        ("n_tokens", _I32), ("n_pages", _I32), ("page_tokens", _I32), ("max_pages", _I32),
        ("layer_begin", _I32), ("n_layers", _I32), ("in_dtype", _I32), ("max_length", _I32),
        ("scale", ctypes.c_float), ("reserved", _I32),
        ("q", _P), ("k", _P), ("v", _P), ("seq_offsets", _P),
        ("k_codes", _P), ("v_codes", _P), ("k_scales", _P), ("v_scales", _P),
        ("pages", _P), ("length", _P),
        ("workspace", _P), ("workspace_bytes", ctypes.c_int64), ("out", _P),
    ]


class SparseArgs(ctypes.Structure):
    _fields_ = [
        ("top_pages", _I32), ("share_tokens", _I32), ("keep_first", _I32), ("keep_last", _I32),
        ("bounds", _P), ("selected", _P),
    ]


class AcceptArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _I32), ("n_nodes", _I32), ("vocab", _I32), ("in_dtype", _I32),
        ("max_path", _I32), ("reserved", _I32), ("logit_stride", ctypes.c_int64),
        ("logits", _P), ("tokens", _P), ("uniform", _P), ("temperature", _P),
        ("path", _P), ("path_len", _P), ("next_token", _P),
        ("workspace", _P), ("workspace_bytes", ctypes.c_int64),
    ]


class LogprobsArgs(ctypes.Structure):
    _fields_ = [
        ("n_rows", _I32), ("vocab", _I32), ("in_dtype", _I32), ("top_k", _I32), ("n_given", _I32),
        ("reserved", _I32), ("logit_stride", ctypes.c_int64),
        ("logits", _P), ("given", _P), ("given_logp", _P), ("top_token", _P), ("top_logp", _P),
        ("entropy", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_int64),
    ]


class PagesArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _I32), ("n_tokens", _I32), ("n_pages", _I32), ("page_tokens", _I32),
        ("max_pages", _I32), ("reserved", _I32),
        ("seq_offsets", _P), ("length", _P), ("pages", _P), ("refs", _P), ("missing", _P),
        ("slots", _P), ("positions", _P), ("depth", _P),
        ("workspace", _P), ("workspace_bytes", ctypes.c_int64),
    ]


_lib = None


# A host-only build of the library's plain C++ parts (schedule, draft-tree builder, commit
# bookkeeping) with AddressSanitizer and UndefinedBehaviorSanitizer (build_host_san.py): when
# this variable names it, lib() loads it instead, for host-side tests; device entry points are
# then absent and torch is not imported.
HOST_LIB_ENV = "GDN_TREE_HOST_LIB"


def host_only() -> bool:
    return bool(os.environ.get(HOST_LIB_ENV))


def _prototypes():
    VA, CA, PA = ctypes.POINTER(VerifyArgs), ctypes.POINTER(ConvArgs), ctypes.POINTER(PrefillArgs)
    KA, AA = ctypes.POINTER(KvArgs), ctypes.POINTER(AcceptArgs)
    GA = ctypes.POINTER(PagesArgs)
    SA, LA = ctypes.POINTER(SparseArgs), ctypes.POINTER(LogprobsArgs)
    return {
        "gdn_last_error": (ctypes.c_char_p, []),
        "gdn_schedule_words": (ctypes.c_size_t, [_I32, _I32]),
        "gdn_hld_schedule": (_I32, [_I32P, _I32P, _I32, _I32P, ctypes.c_size_t]),
        "gdn_ddtree_build": (_I32, [_FP, _I32P, _I32P, _I32, _I32, _I32, _I32, ctypes.c_float,
                                    _I32, _I32P, _I32P, _I32P, _I32P, _FP, _I32P]),
        "gdn_verify_workspace_bytes": (ctypes.c_size_t, [_I32P, _I32, _I32, _I32]),
        "gdn_tree_verify": (_I32, [VA, _I32P, _P, _P]),
        "gdn_tree_verify_noalloc": (_I32, [VA, _I32P, _P, _P]),
        "gdn_tree_verify_wave": (_I32, [VA, _I32P, _P, _I32, _P]),
        "gdn_tree_verify_wave_timed": (_I32, [VA, _I32P, _P, _I32, _P, _P, _P]),
        "gdn_tree_verify_ut": (_I32, [VA, _I32P, _P, _P]),
        "gdn_tree_verify_ut_timed": (_I32, [VA, _I32P, _P, _P, _P, _P]),
        "gdn_prefill": (_I32, [PA, _I32P, _P]),
        "gdn_prefill_timed": (_I32, [PA, _I32P, _P, _P, _P]),
        "gdn_tree_conv_verify": (_I32, [VA, CA, _I32P, _P, _P]),
        "gdn_tree_conv_verify_timed": (_I32, [VA, CA, _I32P, _P, _P, _P, _P]),
        "gdn_tree_conv": (_I32, [CA, _I32P, _P, _P]),
        "gdn_commit_path": (_I32, [_I32P, _I32P, _I32P, _P, _P, VA, CA, _I32P, _I32P, _I32, _P]),
        "gdn_compact_factors": (_I32, [_P, _P, ctypes.c_int64, _P, _P, _I32, _P]),
        "gdn_flush": (_I32, [VA, CA, _I32P, _P]),
        "gdn_kv_append": (_I32, [KA, _I32P, _P]),
        "gdn_kv_commit": (_I32, [KA, _I32P, _P, _I32, _P, _P, _P]),
        "gdn_kv_read": (_I32, [KA, _I32P, _P, _P]),
        "gdn_attention_workspace_bytes": (ctypes.c_size_t, [KA, _I32P]),
        "gdn_attention": (_I32, [KA, _I32P, _P]),
        "gdn_tree_attention": (_I32, [KA, _I32P, _P, _P]),
        "gdn_kv_bounds": (_I32, [KA, SA, _I32P, _P]),
        "gdn_kv_select": (_I32, [KA, SA, _I32P, _P]),
        "gdn_sparse_workspace_bytes": (ctypes.c_size_t, [KA, SA, _I32P]),
        "gdn_sparse_attention": (_I32, [KA, SA, _I32P, _P]),
        "gdn_sparse_tree_attention": (_I32, [KA, SA, _I32P, _P, _P]),
        "gdn_accept_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
        "gdn_tree_accept": (_I32, [AA, _I32P, _P, _P]),
        "gdn_logprobs_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
        "gdn_token_logprobs": (_I32, [LA, _P]),
        "gdn_pages_workspace_bytes": (ctypes.c_size_t, [GA]),
        "gdn_kv_reserve": (_I32, [GA, _P]),
        "gdn_kv_release": (_I32, [GA, _P, _P]),
    }


def lib() -> ctypes.CDLL:
    """Load the HIP library (after torch, so the HIP runtime is shared), or the sanitized
    host-only build named by GDN_TREE_HOST_LIB."""
    global _lib
    if _lib is not None:
        return _lib
    host = os.environ.get(HOST_LIB_ENV)
    if host:
        L = ctypes.CDLL(host)
    else:
        import torch  # noqa: F401  -- must precede the library: one HIP runtime per process
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gated_deltanet_tree_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _prototypes().items():
        if host and not hasattr(L, name):
            continue  # device entry points are not in the host-only build
        fn = getattr(L, name)
        fn.restype = res
        if args:
            fn.argtypes = args
    _lib = L
    return L


def _check(status: int, where: str):
    if status != 0:
        raise GdnError(status, where, lib().gdn_last_error().decode())


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int32)


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(_I32P)


def _dev(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    import torch
    # the current stream's handle without an object around it: 0.4 us, not 2.5, of a call's 6.5
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


# ------------------------------------------------------------------------------------
# schedule (host)
# ------------------------------------------------------------------------------------

def schedule_words(n_seqs: int, n_nodes: int) -> int:
    return int(lib().gdn_schedule_words(n_seqs, n_nodes))


def hld_schedule(parents) -> np.ndarray:
    """Schedule image (int32) of a batch of trees given as a list of local parent arrays."""
    parents = [_i32(p) for p in parents]
    seq_offsets = _i32(np.concatenate([[0], np.cumsum([len(p) for p in parents])]))
    flat = _i32(np.concatenate(parents)) if parents else np.zeros(1, dtype=np.int32)
    n_words = schedule_words(len(parents), int(seq_offsets[-1]))
    image = np.zeros(max(n_words, IMAGE_HEADER + 3), dtype=np.int32)
    _check(lib().gdn_hld_schedule(_ptr(flat), _ptr(seq_offsets), len(parents), _ptr(image),
                                  image.size), "gdn_hld_schedule")
    return image


def schedule_view(image: np.ndarray) -> dict:
    """Named views of a schedule image, following the layout in gdn_tree.h."""
    S, T = int(image[1]), int(image[2])
    n_chains, n_waves = int(image[3]), int(image[4])
    o = IMAGE_HEADER
    seq = image[o:o + S + 1]
    o += S + 1
    wave = image[o:o + n_waves + 1]
    o += T + 1
    chain = image[o:o + n_chains + 1]
    o += T + 1
    fields = {}
    for name in ("chain_nodes", "chain_seq", "chain_src", "node_store", "node_parent",
                 "node_depth"):
        fields[name] = image[o:o + T]
        o += T
    fields["chain_seq"] = fields["chain_seq"][:n_chains]
    fields["chain_src"] = fields["chain_src"][:n_chains]
    ut = None
    if int(image[8]) >= 0:  # tree-masked verify plan
        rec_base = image[o:o + S + 1]
        o += S + 1
        node_rec = image[o:o + T]
        o += T
        lv_base = image[o:o + S + 1]
        o += S + 1
        lvn = image[o:o + int(lv_base[-1])]
        o += T + S
        lvnode = image[o:o + T]
        o += T
        rec_anc = image[o:o + int(rec_base[-1])]
        ut = dict(records=int(image[8]), max_records=int(image[9]), max_levels=int(image[10]),
                  rec_base=rec_base, node_rec=node_rec, lv_base=lv_base, lvn=lvn,
                  lvnode=lvnode, rec_anc=rec_anc)
    return dict(n_seqs=S, n_nodes=T, n_chains=n_chains, n_waves=n_waves,
                n_boundaries=int(image[5]), max_chain_len=int(image[6]), max_tree=int(image[7]),
                seq_offsets=seq, wave_offsets=wave, chain_offsets=chain, ut_plan=ut, **fields)


def ddtree_build(logp, tokens=None, root_tokens=None, budget=22, tau=6.0, chain_seed=True):
    """Best-first draft trees of a batch: logp [B][L][K] (or [L][K]) fp32 log-probabilities,
    tokens of the same shape (optional).  Returns a list of dicts parent/depth/rank/score
    (and token) per tree, each cut to its node count."""
    lp = np.ascontiguousarray(logp, dtype=np.float32)
    single = lp.ndim == 2
    if single:
        lp = lp[None]
    B, L, K = lp.shape
    tk = None if tokens is None else np.ascontiguousarray(tokens, dtype=np.int32).reshape(B, L, K)
    rt = None if root_tokens is None else _i32(np.reshape(root_tokens, (B,)))
    out = {name: np.full((B, budget), -1, dtype=np.int32) for name in ("parent", "depth", "rank",
                                                                        "token")}
    sc = np.zeros((B, budget), dtype=np.float32)
    n = np.zeros(B, dtype=np.int32)
    fp = lambda a: a.ctypes.data_as(_FP)  # noqa: E731
    _check(lib().gdn_ddtree_build(fp(lp), None if tk is None else _ptr(tk),
                                  None if rt is None else _ptr(rt), B, L, K, budget,
                                  ctypes.c_float(tau), int(bool(chain_seed)), _ptr(out["parent"]),
                                  _ptr(out["depth"]), _ptr(out["rank"]),
                                  None if tk is None else _ptr(out["token"]), fp(sc), _ptr(n)),
           "gdn_ddtree_build")
    trees = []
    for b in range(B):
        m = int(n[b])
        t = {k: v[b, :m].copy() for k, v in out.items() if k != "token" or tk is not None}
        t["score"] = sc[b, :m].copy()
        trees.append(t)
    return trees[0] if single else trees


def verify_workspace_bytes(image: np.ndarray, n_heads: int, head_dim: int, n_layers: int) -> int:
    """Workspace bytes of the chain verify (boundary states) for this schedule."""
    return int(lib().gdn_verify_workspace_bytes(_ptr(image), n_heads, head_dim, n_layers))





# ------------------------------------------------------------------------------------
# device calls
# ------------------------------------------------------------------------------------

@dataclass
class Layers:
    """Device buffers of a stack of GDN layers for one batch of sequences (torch tensors).

    Shapes: state [Ly,S,H,d,d]; bank_k/bank_u [2][Ly,S,H,max_nodes,d]; bank_lg
    [2][Ly,S,H,max_nodes]; conv_state [Ly,S,Cch,3]; bank_x [2][Ly,S,max_nodes,Cch];
    bank_x holds the raw conv inputs in their own dtype (bf16 or fp32);
    role, pending [S] int32 (device) with host mirrors role_host, pending_host;
    pending_rows [S,max_nodes] int32 (device): the bank row of each pending factor.
    """
    state: object
    bank_k: list
    bank_u: list
    bank_lg: list
    role: object
    pending: object
    role_host: np.ndarray
    pending_host: np.ndarray
    pending_rows: object = None
    conv_state: object = None
    bank_x: list = None


def _need(t, n, what):
    """Reject a tensor that is smaller than the call will address (or not contiguous)."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{what} holds {t.numel()} elements, the call addresses {n}")


def verify_args(image, layers: Layers, q, k, v, beta, gate, out, workspace,
                layer_begin=0, n_layers=1, max_nodes=None) -> VerifyArgs:
    import torch
    S, T = int(image[1]), int(image[2])
    Ly_end = layer_begin + n_layers
    H, d = int(layers.state.shape[2]), int(layers.state.shape[3])
    Nm = int(layers.bank_lg[0].shape[-1]) if max_nodes is None else max_nodes
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _need(t, Ly_end * T * H * d, name)
    _need(beta, Ly_end * T * H, "beta")
    _need(gate, Ly_end * T * H, "gate")
    _need(layers.state, Ly_end * S * H * d * d, "state")
    for i in range(2):
        _need(layers.bank_k[i], Ly_end * S * H * Nm * d, "bank_k")
        _need(layers.bank_u[i], Ly_end * S * H * Nm * d, "bank_u")
        _need(layers.bank_lg[i], Ly_end * S * H * Nm, "bank_lg")
    _need(layers.role, S, "role")
    _need(layers.pending, S, "pending")
    _need(layers.pending_rows, S * Nm, "pending_rows")
    _need(workspace, 0, "workspace")
    a = VerifyArgs()
    # kept for the size check of the chain entry points
    a.ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.sizes = (H, d, n_layers)
    a.n_seqs, a.n_nodes = int(image[1]), int(image[2])
    a.n_heads, a.head_dim = int(layers.state.shape[2]), int(layers.state.shape[3])
    a.max_nodes = int(layers.bank_lg[0].shape[-1]) if max_nodes is None else max_nodes
    a.layer_begin, a.n_layers = layer_begin, n_layers
    ref = q if q is not None else beta  # the fused conv -> verify call passes no q/k/v
    a.in_dtype = GDN_BF16 if (ref is not None and ref.dtype == torch.bfloat16) else GDN_F32
    a.q, a.k, a.v, a.beta, a.gate = (_dev(t) for t in (q, k, v, beta, gate))
    a.state = _dev(layers.state)
    for i in range(2):
        a.bank_k[i] = _dev(layers.bank_k[i])
        a.bank_u[i] = _dev(layers.bank_u[i])
        a.bank_lg[i] = _dev(layers.bank_lg[i])
    a.role, a.pending_len = _dev(layers.role), _dev(layers.pending)
    a.pending_rows = _dev(layers.pending_rows)
    a.workspace, a.out = _dev(workspace), _dev(out)
    return a


def conv_args(image, layers: Layers, x, weight, out, layer_begin=0, n_layers=1,
              max_nodes=None) -> ConvArgs:
    import torch
    S, T = int(image[1]), int(image[2])
    Ly_end = layer_begin + n_layers
    C = int(layers.conv_state.shape[2])
    Nm = int(layers.bank_x[0].shape[2]) if max_nodes is None else max_nodes
    _need(x, Ly_end * T * C, "x")
    _need(out, Ly_end * T * C, "conv out")
    _need(weight, Ly_end * C * 4, "weight")
    _need(layers.conv_state, Ly_end * S * C * 3, "conv_state")
    for i in range(2):
        _need(layers.bank_x[i], Ly_end * S * Nm * C, "bank_x")
    a = ConvArgs()
    a.n_seqs, a.n_nodes = int(image[1]), int(image[2])
    a.channels, a.width = int(layers.conv_state.shape[2]), 4
    a.max_nodes = int(layers.bank_x[0].shape[2]) if max_nodes is None else max_nodes
    a.layer_begin, a.n_layers = layer_begin, n_layers
    # the conv bank keeps the raw inputs in their own dtype: x (when given) must match it
    bank_bf16 = layers.bank_x[0].dtype == torch.bfloat16
    if x is not None and (x.dtype == torch.bfloat16) != bank_bf16:
        raise ValueError(f"x is {x.dtype} but the conv bank holds {layers.bank_x[0].dtype}: "
                         "allocate the layers with conv_dtype matching the conv inputs")
    a.in_dtype = GDN_BF16 if bank_bf16 else GDN_F32
    a.x, a.weight, a.out = _dev(x), _dev(weight), _dev(out)
    a.conv_state = _dev(layers.conv_state)
    a.bank_x[0], a.bank_x[1] = _dev(layers.bank_x[0]), _dev(layers.bank_x[1])
    _need(layers.pending_rows, S * Nm, "pending_rows")
    a.role, a.pending_len = _dev(layers.role), _dev(layers.pending)
    a.pending_rows = _dev(layers.pending_rows)
    return a


def _need_ws(args: VerifyArgs, image: np.ndarray):
    """The chain verify writes boundary states into the workspace: check its size."""
    if args.q is None:
        return
    H, d, n_layers = args.sizes
    need = verify_workspace_bytes(image, H, d, n_layers)
    if need and args.ws_bytes < need:
        raise ValueError(f"workspace holds {args.ws_bytes} bytes, the call needs {need}")


def tree_verify(args: VerifyArgs, image: np.ndarray, dev_image, stream=None):
    _need_ws(args, image)
    _check(lib().gdn_tree_verify(ctypes.byref(args), _ptr(image), _dev(dev_image),
                                 _stream(stream)), "gdn_tree_verify")


def tree_verify_noalloc(args: VerifyArgs, image: np.ndarray, dev_image, stream=None):
    """gdn_tree_verify with the boundary states in the library's fixed device scratch
    (args.workspace is ignored); allocates nothing."""
    _check(lib().gdn_tree_verify_noalloc(ctypes.byref(args), _ptr(image), _dev(dev_image),
                                         _stream(stream)), "gdn_tree_verify_noalloc")


def tree_verify_wave(args: VerifyArgs, image: np.ndarray, dev_image, wave: int, stream=None):
    _need_ws(args, image)
    _check(lib().gdn_tree_verify_wave(ctypes.byref(args), _ptr(image), _dev(dev_image), wave,
                                      _stream(stream)), "gdn_tree_verify_wave")


def tree_verify_wave_timed(args: VerifyArgs, image: np.ndarray, dev_image, wave: int,
                           start: "HipEvent", stop: "HipEvent", stream=None):
    _need_ws(args, image)
    _check(lib().gdn_tree_verify_wave_timed(ctypes.byref(args), _ptr(image), _dev(dev_image), wave,
                                            start.handle, stop.handle, _stream(stream)),
           "gdn_tree_verify_wave_timed")


def tree_verify_ut(args: VerifyArgs, image: np.ndarray, dev_image, stream=None):
    _check(lib().gdn_tree_verify_ut(ctypes.byref(args), _ptr(image), _dev(dev_image),
                                    _stream(stream)), "gdn_tree_verify_ut")


def tree_verify_ut_timed(args: VerifyArgs, image: np.ndarray, dev_image, start: "HipEvent",
                         stop: "HipEvent", stream=None):
    _check(lib().gdn_tree_verify_ut_timed(ctypes.byref(args), _ptr(image), _dev(dev_image),
                                          start.handle, stop.handle, _stream(stream)),
           "gdn_tree_verify_ut_timed")


def tree_conv_verify(vargs: VerifyArgs, cargs: ConvArgs, image: np.ndarray, dev_image,
                     stream=None):
    """Fused conv -> SiLU -> unit-length q/k -> tree-masked verify (gdn_tree_conv_verify);
    vargs carries no q/k/v, cargs no conv output."""
    _check(lib().gdn_tree_conv_verify(ctypes.byref(vargs), ctypes.byref(cargs), _ptr(image),
                                      _dev(dev_image), _stream(stream)), "gdn_tree_conv_verify")


def tree_conv_verify_timed(vargs: VerifyArgs, cargs: ConvArgs, image: np.ndarray, dev_image,
                           start: "HipEvent", stop: "HipEvent", stream=None):
    _check(lib().gdn_tree_conv_verify_timed(ctypes.byref(vargs), ctypes.byref(cargs),
                                            _ptr(image), _dev(dev_image), start.handle,
                                            stop.handle, _stream(stream)),
           "gdn_tree_conv_verify_timed")


def prefill_args(host_offsets, dev_offsets, q, k, v, beta, gate, state, out, layer_begin=0,
                 n_layers=1):
    """Arguments of gdn_prefill; q/k/v [Ly][T][H][d], beta/gate [Ly][T][H], state
    [Ly][S][H][d][d], out [Ly][T][H][d] (torch tensors), offsets [S+1] (numpy + device)."""
    import torch
    host_offsets = _i32(host_offsets)
    S, T = len(host_offsets) - 1, int(host_offsets[-1])
    H, d = int(state.shape[2]), int(state.shape[3])
    Ly_end = layer_begin + n_layers
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _need(t, Ly_end * T * H * d, name)
    _need(beta, Ly_end * T * H, "beta")
    _need(gate, Ly_end * T * H, "gate")
    _need(state, Ly_end * S * H * d * d, "state")
    _need(dev_offsets, S + 1, "seq_offsets")
    a = PrefillArgs()
    a.n_seqs, a.n_heads, a.head_dim, a.n_tokens = S, H, d, T
    a.layer_begin, a.n_layers = layer_begin, n_layers
    a.in_dtype = GDN_BF16 if q.dtype == torch.bfloat16 else GDN_F32
    a.q, a.k, a.v, a.beta, a.gate = (_dev(t) for t in (q, k, v, beta, gate))
    a.seq_offsets, a.state, a.out = _dev(dev_offsets), _dev(state), _dev(out)
    a.host_offsets = host_offsets
    return a


def prefill(args: PrefillArgs, stream=None):
    _check(lib().gdn_prefill(ctypes.byref(args), _ptr(args.host_offsets), _stream(stream)),
           "gdn_prefill")


def prefill_timed(args: PrefillArgs, start: "HipEvent", stop: "HipEvent", stream=None):
    _check(lib().gdn_prefill_timed(ctypes.byref(args), _ptr(args.host_offsets), start.handle,
                                   stop.handle, _stream(stream)), "gdn_prefill_timed")


class HipEvent:
    """A timing-enabled hipEvent_t from the process's HIP runtime (the one torch loaded)."""
    _hip = None

    @classmethod
    def _runtime(cls):
        if cls._hip is None:
            lib()
            h = ctypes.CDLL("libamdhip64.so.7")
            h.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
            h.hipEventDestroy.argtypes = [ctypes.c_void_p]
            h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                              ctypes.c_void_p]
            cls._hip = h
        return cls._hip

    def __init__(self):
        self.handle = ctypes.c_void_p()
        rc = self._runtime().hipEventCreate(ctypes.byref(self.handle))
        if rc != 0:
            raise RuntimeError(f"hipEventCreate failed: {rc}")

    def elapsed_ms(self, stop: "HipEvent") -> float:
        ms = ctypes.c_float()
        rc = self._runtime().hipEventElapsedTime(ctypes.byref(ms), self.handle, stop.handle)
        if rc != 0:
            raise RuntimeError(f"hipEventElapsedTime failed: {rc}")
        return ms.value

    def __del__(self):
        if self._hip is not None and self.handle:
            self._hip.hipEventDestroy(self.handle)


def tree_conv(args: ConvArgs, image: np.ndarray, dev_image, stream=None):
    _check(lib().gdn_tree_conv(ctypes.byref(args), _ptr(image), _dev(dev_image),
                               _stream(stream)), "gdn_tree_conv")


def pack_paths(paths):
    flat = _i32(np.concatenate([np.asarray(p, dtype=np.int32) for p in paths])) \
        if any(len(p) for p in paths) else np.zeros(1, dtype=np.int32)
    offsets = _i32(np.concatenate([[0], np.cumsum([len(p) for p in paths])]))
    return flat, offsets


COMMIT_COMPACT, COMMIT_ROW_MAP = 0, 1


def commit_path(image, paths, layers: Layers, vargs: VerifyArgs, cargs: ConvArgs | None,
                dev_paths=None, dev_offsets=None, stream=None, mode=COMMIT_ROW_MAP):
    """Accept one root path per sequence (local ids); updates layers.role/pending/pending_rows
    (device on the stream, host mirrors now).  dev_paths/dev_offsets default to fresh
    uploads.  mode: COMMIT_ROW_MAP (no copy) or COMMIT_COMPACT (branched paths gathered into
    path order)."""
    import torch
    flat, offsets = pack_paths(paths)
    if dev_paths is None:
        dev_paths = torch.from_numpy(flat).to(layers.role.device)
        dev_offsets = torch.from_numpy(offsets).to(layers.role.device)
    _check(lib().gdn_commit_path(
        _ptr(image), _ptr(flat), _ptr(offsets), _dev(dev_paths), _dev(dev_offsets),
        ctypes.byref(vargs), ctypes.byref(cargs) if cargs is not None else None,
        _ptr(layers.role_host), _ptr(layers.pending_host), int(mode), _stream(stream)),
        "gdn_commit_path")
    return dev_paths, dev_offsets


def compact_factors(src, dst, row_elems: int, src_rows, dst_rows, stream=None):
    _check(lib().gdn_compact_factors(_dev(src), _dev(dst), row_elems, _dev(src_rows),
                                     _dev(dst_rows), int(src_rows.numel()), _stream(stream)),
           "gdn_compact_factors")


def flush(vargs: VerifyArgs, cargs: ConvArgs | None, layers: Layers, stream=None):
    _check(lib().gdn_flush(ctypes.byref(vargs), ctypes.byref(cargs) if cargs is not None else None,
                           _ptr(layers.pending_host), _stream(stream)), "gdn_flush")


def alloc_layers(n_layers, n_seqs, n_heads, head_dim, max_nodes, channels=0, device="cuda",
                 conv_dtype="f32"):
    """Zero-initialised device buffers for `n_layers` layers (torch.empty/zeros on device);
    conv_dtype ("f32" or "bf16") is the dtype of the conv inputs, which the conv bank keeps."""
    import torch
    f = dict(device=device, dtype=torch.float32)
    Ly, S, H, d, Nm = n_layers, n_seqs, n_heads, head_dim, max_nodes
    lay = Layers(
        state=torch.zeros((Ly, S, H, d, d), **f),
        bank_k=[torch.zeros((Ly, S, H, Nm, d), **f) for _ in range(2)],
        bank_u=[torch.zeros((Ly, S, H, Nm, d), **f) for _ in range(2)],
        bank_lg=[torch.zeros((Ly, S, H, Nm), **f) for _ in range(2)],
        role=torch.zeros(S, device=device, dtype=torch.int32),
        pending=torch.zeros(S, device=device, dtype=torch.int32),
        role_host=np.zeros(S, dtype=np.int32),
        pending_host=np.zeros(S, dtype=np.int32),
        pending_rows=torch.zeros((S, Nm), device=device, dtype=torch.int32),
    )
    if channels:
        lay.conv_state = torch.zeros((Ly, S, channels, 3), **f)
        xdt = torch.bfloat16 if conv_dtype == "bf16" else torch.float32
        lay.bank_x = [torch.zeros((Ly, S, Nm, channels), device=device, dtype=xdt)
                      for _ in range(2)]
    return lay


# ------------------------------------------------------------------------------------
# 4-bit key/value cache, its attention, and the acceptance of a draft tree
# ------------------------------------------------------------------------------------

@dataclass
class KvCache:
    """Device buffers of the 4-bit paged key/value cache of a stack of attention layers (torch
    tensors; the pools' inner layout is the library's).

    Shapes: k_codes, v_codes uint8 [Ly][n_pages][Hkv][page_tokens * d / 2]; k_scales, v_scales uint8
    [Ly][n_pages][Hkv][page_tokens * d / 32]; pages int32 [S][max_pages] (an id outside
    [0, n_pages) is a page that is not there); length int32 [S], the committed tokens.
    """
    k_codes: object
    k_scales: object
    v_codes: object
    v_scales: object
    pages: object
    length: object
    page_tokens: int


def alloc_kv_cache(n_layers, n_seqs, n_kv_heads, head_dim, n_pages, page_tokens, max_pages,
                   device="cuda") -> KvCache:
    """Zero-initialised pools, no pages assigned (-1) and nothing committed."""
    import torch
    u8 = dict(device=device, dtype=torch.uint8)
    i32 = dict(device=device, dtype=torch.int32)
    codes = (n_layers, n_pages, n_kv_heads, page_tokens * head_dim // 2)
    scales = (n_layers, n_pages, n_kv_heads, page_tokens * head_dim // 32)
    return KvCache(torch.zeros(codes, **u8), torch.zeros(scales, **u8), torch.zeros(codes, **u8),
                   torch.zeros(scales, **u8), torch.full((n_seqs, max_pages), -1, **i32),
                   torch.zeros(n_seqs, **i32), page_tokens)


def _typed(t, dtype, what):
    if t is not None and t.dtype != dtype:
        raise ValueError(f"{what} is {t.dtype}, expected {dtype}")


def _devices(tensors):
    return {t.device for t in tensors if t is not None}


def _same_device(args, more, what):
    """Reject tensors on the host or on several devices; the launch goes to the current one."""
    import torch
    devs = args.devices if not more else args.devices | _devices(more)
    if len(devs) == 1 and args.device_index >= 0 and args.device_index == torch.cuda.current_device():
        return
    if any(d.type != "cuda" for d in devs):
        raise ValueError(f"{what}: tensors must be in GPU memory, got {sorted(map(str, devs))}")
    raise ValueError(f"{what}: tensors on {sorted(map(str, devs))}, the current device is "
                     f"cuda:{torch.cuda.current_device()}")


def _keep(args, tensors):
    """Keeps an argument struct's tensors alive with it, and where they are."""
    args.tensors, args.devices = tensors, _devices(tensors)
    (d,) = args.devices if len(args.devices) == 1 else (None,)
    args.device_index = d.index if d is not None and d.type == "cuda" else -1


def kv_args(cache: KvCache, host_offsets, dev_offsets, q=None, k=None, v=None, out=None,
            workspace=None, scale=None, max_length=0, layer_begin=0, n_layers=1) -> KvArgs:
    """Arguments of the cache calls: k, v [Ly][T][Hkv][d] for kv_append, kv_commit and kv_read
    (which writes them), q, out [Ly][T][Hq][d] for the attention (bf16 or fp32, all alike); offsets
    [S+1] (numpy + device): new tokens of sequence b are rows offsets[b] .. offsets[b+1].
    scale (> 0) defaults to 1 / sqrt(d); max_length (0: the page table's capacity) is the longest
    length + new tokens expected, which sizes the attention's split and workspace."""
    import torch
    host_offsets = _i32(host_offsets)
    S, T = len(host_offsets) - 1, int(host_offsets[-1])
    Ly, n_pages, Hkv = (int(x) for x in cache.k_codes.shape[:3])
    pt = int(cache.page_tokens)
    d = int(cache.k_codes.shape[3]) * 2 // max(pt, 1)
    Ly_end = layer_begin + n_layers
    if layer_begin < 0 or n_layers < 1 or Ly_end > Ly:
        raise ValueError(f"layers {layer_begin} .. {Ly_end - 1} of a cache of {Ly}")
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        t = getattr(cache, name)
        _typed(t, torch.uint8, name)
        _need(t, Ly * n_pages * Hkv * pt * d // (2 if name.endswith("codes") else 32), name)
    _typed(cache.pages, torch.int32, "pages")
    _typed(cache.length, torch.int32, "length")
    if cache.pages.dim() != 2 or cache.pages.shape[0] < S:
        raise ValueError(f"pages is {tuple(cache.pages.shape)}, expected [{S}][max_pages]")
    _need(cache.pages, S, "pages")
    _need(cache.length, S, "length")
    _typed(dev_offsets, torch.int32, "seq_offsets")
    _need(dev_offsets, S + 1, "seq_offsets")
    Hq = Hkv
    if q is not None:
        if q.dim() != 4 or int(q.shape[3]) != d:
            raise ValueError(f"q is {tuple(q.shape)}, expected [layers][tokens][heads][{d}]")
        Hq = int(q.shape[2])
    for name, t, h in (("q", q, Hq), ("out", out, Hq), ("k", k, Hkv), ("v", v, Hkv)):
        _need(t, Ly_end * T * h * d, name)
        if t is None or t.dim() != 4:
            continue
        if (int(t.shape[2]), int(t.shape[3])) != (h, d):
            raise ValueError(f"{name} is {tuple(t.shape)}, expected [layers][tokens][{h}][{d}]")
        if Ly_end > 1 and int(t.shape[1]) != T:
            raise ValueError(f"{name} is {tuple(t.shape)}: a layer's rows must be the {T} of the offsets")
    rows = [t for t in (q, out, k, v) if t is not None]
    if any(t.dtype not in (torch.bfloat16, torch.float32) or t.dtype != rows[0].dtype
           for t in rows):
        raise ValueError(f"q, out, k and v must all be bf16 or all fp32, got "
                         f"{[str(t.dtype) for t in rows]}")
    _need(workspace, 0, "workspace")
    a = KvArgs()
    _keep(a, (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.pages,
              cache.length, dev_offsets, q, k, v, out, workspace))
    a.host_offsets, a.host_ptr = host_offsets, _ptr(host_offsets)
    a.n_seqs, a.n_heads, a.n_kv_heads, a.head_dim = S, Hq, Hkv, d
    a.n_tokens, a.n_pages, a.page_tokens = T, n_pages, pt
    a.max_pages = int(cache.pages.shape[1])
    a.layer_begin, a.n_layers, a.max_length = layer_begin, n_layers, int(max_length)
    a.in_dtype = GDN_BF16 if rows and rows[0].dtype == torch.bfloat16 else GDN_F32
    a.scale = float(d) ** -0.5 if scale is None else float(scale)
    a.q, a.k, a.v, a.out = _dev(q), _dev(k), _dev(v), _dev(out)
    a.seq_offsets = _dev(dev_offsets)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales", "pages", "length"):
        setattr(a, name, _dev(getattr(cache, name)))
    a.workspace = _dev(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return a


def kv_append(args: KvArgs, stream=None):
    """Quantises row i of every sequence into its slot length + i."""
    _same_device(args, (), "kv_append")
    _check(lib().gdn_kv_append(ctypes.byref(args), args.host_ptr, _stream(stream)),
           "gdn_kv_append")


def kv_commit(args: KvArgs, rows, counts, new_length, stream=None):
    """Commits the accepted rows: row rows[b][i], i < counts[b], goes to slot length + i (rows
    None: they already sit there), and new_length = length + counts, which may be the cache's
    length itself (or counts, nothing else among the inputs); all layers in one call.  rows, counts:
    int32 tensors as tree_accept writes path and path_len."""
    import torch
    for t, n, what in ((counts, args.n_seqs, "counts"), (new_length, args.n_seqs, "new_length")):
        _typed(t, torch.int32, what)
        _need(t, n, what)
    width = 0
    if rows is not None:
        _typed(rows, torch.int32, "rows")
        if rows.dim() != 2 or rows.shape[0] < args.n_seqs:
            raise ValueError(f"rows is {tuple(rows.shape)}, expected [{args.n_seqs}][width]")
        _need(rows, 0, "rows")
        width = int(rows.shape[1])
    _same_device(args, (rows, counts, new_length), "kv_commit")
    _check(lib().gdn_kv_commit(ctypes.byref(args), args.host_ptr, _dev(rows), width,
                               _dev(counts), _dev(new_length), _stream(stream)), "gdn_kv_commit")


def kv_read(args: KvArgs, begin=None, stream=None):
    """Stored values of slots begin + i (default: length + i) into the args' k and v."""
    import torch
    _typed(begin, torch.int32, "begin")
    _need(begin, args.n_seqs, "begin")
    _same_device(args, (begin,), "kv_read")
    _check(lib().gdn_kv_read(ctypes.byref(args), args.host_ptr, _dev(begin),
                             _stream(stream)), "gdn_kv_read")


def attention_workspace_bytes(args: KvArgs) -> int:
    """Workspace bytes of attention / tree_attention with these sizes (0: none needed)."""
    return int(lib().gdn_attention_workspace_bytes(ctypes.byref(args), args.host_ptr))


def attention(args: KvArgs, stream=None):
    """Causal attention of the new tokens over the cache (they must have been appended)."""
    _same_device(args, (), "attention")
    _check(lib().gdn_attention(ctypes.byref(args), args.host_ptr, _stream(stream)),
           "gdn_attention")


def tree_attention(args: KvArgs, image: np.ndarray, dev_image, stream=None):
    """Attention of draft-tree nodes: the committed slots, a node's ancestors and itself."""
    _same_device(args, (dev_image,), "tree_attention")
    _check(lib().gdn_tree_attention(ctypes.byref(args), _ptr(image), _dev(dev_image),
                                    _stream(stream)), "gdn_tree_attention")


def alloc_kv_refs(cache: KvCache):
    """References of a cache's pages, int32 [n_pages]: how many of its table entries hold each."""
    import torch
    n_pages = int(cache.k_codes.shape[1])
    held = cache.pages[(cache.pages >= 0) & (cache.pages < n_pages)].long()
    return torch.bincount(held, minlength=n_pages).to(torch.int32)


def pages_args(pages, length, refs, page_tokens, host_offsets, dev_offsets, missing=None, slots=None,
               positions=None, depth=None, workspace=None) -> PagesArgs:
    """Arguments of kv_reserve and kv_release: a cache's pages [S][max_pages], length [S] and page_tokens,
    the pool's refs [n_pages] (all int32), offsets [S+1] (numpy + device) of the new tokens; outputs missing
    [S] int32, slots [T] int64 and positions [T] int32, each optional; depth [T] int32 (a draft tree's
    node_depth) for the positions."""
    import torch
    host_offsets = _i32(host_offsets)
    S, T = len(host_offsets) - 1, int(host_offsets[-1])
    if host_offsets[0] != 0 or (np.diff(host_offsets) < 0).any():
        raise ValueError("offsets must start at 0 and not decrease")
    if pages.dim() != 2 or pages.shape[0] < S:
        raise ValueError(f"pages is {tuple(pages.shape)}, expected [{S}][max_pages]")
    for name, t, n, dt in (("pages", pages, S, torch.int32), ("length", length, S, torch.int32),
                           ("refs", refs, 1, torch.int32), ("seq_offsets", dev_offsets, S + 1, torch.int32),
                           ("missing", missing, S, torch.int32), ("slots", slots, T, torch.int64),
                           ("positions", positions, T, torch.int32), ("depth", depth, T, torch.int32)):
        _typed(t, dt, name)
        _need(t, n, name)
    _need(workspace, 0, "workspace")
    a = PagesArgs()
    _keep(a, (pages, length, refs, dev_offsets, missing, slots, positions, depth, workspace))
    a.n_seqs, a.n_tokens, a.n_pages = S, T, int(refs.numel())
    a.page_tokens, a.max_pages = int(page_tokens), int(pages.shape[1])
    a.seq_offsets, a.length, a.pages, a.refs = (_dev(t) for t in (dev_offsets, length, pages, refs))
    a.missing, a.slots, a.positions, a.depth = (_dev(t) for t in (missing, slots, positions, depth))
    a.workspace = _dev(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return a


def pages_workspace_bytes(args: PagesArgs) -> int:
    """Workspace bytes of kv_reserve with these sizes."""
    return int(lib().gdn_pages_workspace_bytes(ctypes.byref(args)))


def kv_reserve(args: PagesArgs, stream=None):
    """Pages for the committed and the new tokens of every sequence, and the new tokens' slots and
    positions; missing counts the entries that are left without."""
    _same_device(args, (), "kv_reserve")
    _check(lib().gdn_kv_reserve(ctypes.byref(args), _stream(stream)), "gdn_kv_reserve")


def kv_release(args: PagesArgs, keep, stream=None):
    """Gives back the pages behind the first keep[b] slots of every sequence (int32 [S])."""
    import torch
    _typed(keep, torch.int32, "keep")
    _need(keep, args.n_seqs, "keep")
    _same_device(args, (keep,), "kv_release")
    _check(lib().gdn_kv_release(ctypes.byref(args), _dev(keep), _stream(stream)), "gdn_kv_release")


def alloc_kv_bounds(cache: KvCache):
    """Zeroed bounds of a cache's pages, bf16 [Ly][n_pages][Hkv][2][d]: what kv_bounds writes."""
    import torch
    Ly, n_pages, Hkv = cache.k_codes.shape[:3]
    d = int(cache.k_codes.shape[3]) * 2 // int(cache.page_tokens)
    return torch.zeros((Ly, n_pages, Hkv, 2, d), device=cache.k_codes.device, dtype=torch.bfloat16)


def sparse_args(args: KvArgs, bounds=None, selected=None, top_pages=0, share_tokens=1, keep_first=0,
                keep_last=0) -> SparseArgs:
    """What sparse attention takes beside kv_args: bounds bf16 [Ly][n_pages][Hkv][2][d] (kv_bounds writes
    them, kv_select reads them) and selected int32 [Ly][T][Hkv][top_pages] (kv_select writes it, the
    attention reads it; a selection's entries stand at its first token).  share_tokens consecutive new
    tokens share a selection, 0: all of a sequence (trees: 0)."""
    import torch
    Ly_end = args.layer_begin + args.n_layers
    _typed(bounds, torch.bfloat16, "bounds")
    _need(bounds, Ly_end * args.n_pages * args.n_kv_heads * 2 * args.head_dim, "bounds")
    _typed(selected, torch.int32, "selected")
    _need(selected, Ly_end * args.n_tokens * args.n_kv_heads * max(int(top_pages), 0), "selected")
    for name, t, tail in (("bounds", bounds, (args.n_pages, args.n_kv_heads, 2, args.head_dim)),
                          ("selected", selected, (args.n_tokens, args.n_kv_heads, int(top_pages)))):
        if t is not None and t.dim() == len(tail) + 1 and tuple(t.shape[1:]) != tail:
            raise ValueError(f"{name} is {tuple(t.shape)}, expected [layers]{list(tail)}")
    x = SparseArgs()
    _keep(x, (bounds, selected))
    x.top_pages, x.share_tokens = int(top_pages), int(share_tokens)
    x.keep_first, x.keep_last = int(keep_first), int(keep_last)
    x.bounds, x.selected = _dev(bounds), _dev(selected)
    return x


def kv_bounds(args: KvArgs, sparse: SparseArgs, stream=None):
    """Bounds of the full pages that the last new tokens before length may have filled (after kv_commit)."""
    _same_device(args, sparse.tensors, "kv_bounds")
    _check(lib().gdn_kv_bounds(ctypes.byref(args), ctypes.byref(sparse), args.host_ptr, _stream(stream)),
           "gdn_kv_bounds")


def sparse_workspace_bytes(args: KvArgs, sparse: SparseArgs) -> int:
    """Workspace bytes of kv_select and the sparse attention with these sizes (0: none needed)."""
    return int(lib().gdn_sparse_workspace_bytes(ctypes.byref(args), ctypes.byref(sparse), args.host_ptr))


def kv_select(args: KvArgs, sparse: SparseArgs, stream=None):
    """Selects the pages each selection of the new tokens attends to, from q and the bounds."""
    _same_device(args, sparse.tensors, "kv_select")
    _check(lib().gdn_kv_select(ctypes.byref(args), ctypes.byref(sparse), args.host_ptr, _stream(stream)),
           "gdn_kv_select")


def sparse_attention(args: KvArgs, sparse: SparseArgs, stream=None):
    """Causal attention over the selected pages and the slots behind the full ones."""
    _same_device(args, sparse.tensors, "sparse_attention")
    _check(lib().gdn_sparse_attention(ctypes.byref(args), ctypes.byref(sparse), args.host_ptr,
                                      _stream(stream)), "gdn_sparse_attention")


def sparse_tree_attention(args: KvArgs, sparse: SparseArgs, image: np.ndarray, dev_image, stream=None):
    """Attention of draft-tree nodes over the selected pages, the slots behind the full ones, a node's
    ancestors and itself."""
    _same_device(args, sparse.tensors + (dev_image,), "sparse_tree_attention")
    _check(lib().gdn_sparse_tree_attention(ctypes.byref(args), ctypes.byref(sparse), _ptr(image),
                                           _dev(dev_image), _stream(stream)), "gdn_sparse_tree_attention")


def accept_workspace_bytes(image: np.ndarray, vocab: int) -> int:
    """Workspace bytes of tree_accept for this schedule and vocabulary."""
    return int(lib().gdn_accept_workspace_bytes(int(image[1]), int(image[2]), vocab))


def accept_args(image: np.ndarray, logits, tokens, uniform, temperature, path, path_len,
                next_token, workspace, vocab=None) -> AcceptArgs:
    """Arguments of tree_accept: logits [T][>= vocab] (bf16 or fp32, rows of any stride, unit
    element stride), tokens [T] int32, uniform [S][max_path] fp32 in [0, 1), temperature [S] fp32;
    outputs path [S][max_path], path_len [S], next_token [S] int32.  vocab defaults to the
    logits' width."""
    import torch
    S, T = int(image[1]), int(image[2])
    if logits.dim() != 2 or logits.shape[0] < T or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits is {tuple(logits.shape)} with strides {tuple(logits.stride())}, "
                         f"expected [{T}][vocab] rows")
    V = int(logits.shape[1]) if vocab is None else int(vocab)
    if V > logits.shape[1]:
        raise ValueError(f"vocab {V} exceeds the logits' width {int(logits.shape[1])}")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits is {logits.dtype}, expected bf16 or fp32")
    if path.dim() != 2 or uniform.dim() != 2 or path.shape[1] != uniform.shape[1]:
        raise ValueError("path and uniform must be [sequences][max_path] alike")
    width = int(path.shape[1])
    for name, t, n, dt in (("tokens", tokens, T, torch.int32),
                           ("uniform", uniform, S * width, torch.float32),
                           ("temperature", temperature, S, torch.float32),
                           ("path", path, S * width, torch.int32),
                           ("path_len", path_len, S, torch.int32),
                           ("next_token", next_token, S, torch.int32)):
        _typed(t, dt, name)
        _need(t, n, name)
    _need(workspace, 0, "workspace")
    a = AcceptArgs()
    _keep(a, (logits, tokens, uniform, temperature, path, path_len, next_token, workspace))
    a.n_seqs, a.n_nodes, a.vocab, a.max_path = S, T, V, width
    a.in_dtype = GDN_BF16 if logits.dtype == torch.bfloat16 else GDN_F32
    a.logit_stride = int(logits.stride(0)) if T > 1 else max(V, int(logits.shape[1]))
    a.logits, a.tokens, a.uniform, a.temperature = (_dev(t) for t in (logits, tokens, uniform,
                                                                      temperature))
    a.path, a.path_len, a.next_token = _dev(path), _dev(path_len), _dev(next_token)
    a.workspace = _dev(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return a


def tree_accept(args: AcceptArgs, image: np.ndarray, dev_image, stream=None):
    """Accepted root path and next token of every tree; path and path_len go to kv_commit as they
    are, and to commit_path from the host."""
    _same_device(args, (dev_image,), "tree_accept")
    _check(lib().gdn_tree_accept(ctypes.byref(args), _ptr(image), _dev(dev_image),
                                 _stream(stream)), "gdn_tree_accept")


# ------------------------------------------------------------------------------------
# log probabilities of rows of logits
# ------------------------------------------------------------------------------------

def logprobs_workspace_bytes(n_rows: int, vocab: int, top_k: int) -> int:
    """Workspace bytes of token_logprobs."""
    return int(lib().gdn_logprobs_workspace_bytes(n_rows, vocab, top_k))


def logprobs_args(logits, given=None, given_logp=None, top_token=None, top_logp=None, entropy=None,
                  workspace=None, vocab=None) -> LogprobsArgs:
    """Arguments of token_logprobs: logits [N][>= vocab] (bf16 or fp32, rows of any stride, unit element
    stride), given [N][M] int32; outputs given_logp [N][M], top_token [N][K] int32, top_logp [N][K],
    entropy [N] (fp32), each optional (given with given_logp, top_token with top_logp).  vocab defaults to
    the logits' width.  With N = trees * positions, top_logp and top_token on the host are ddtree_build's
    logp and tokens."""
    import torch
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1) or \
            (logits.shape[0] > 1 and logits.stride(0) < logits.shape[1]):
        raise ValueError(f"logits is {tuple(logits.shape)} with strides {tuple(logits.stride())}, "
                         "expected [rows][vocab] rows")
    N = int(logits.shape[0])
    V = int(logits.shape[1]) if vocab is None else int(vocab)
    if V > logits.shape[1]:
        raise ValueError(f"vocab {V} exceeds the logits' width {int(logits.shape[1])}")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits is {logits.dtype}, expected bf16 or fp32")
    width = {}
    for name, a, b, da, db in (("given", given, given_logp, torch.int32, torch.float32),
                               ("top_token", top_token, top_logp, torch.int32, torch.float32)):
        if (a is None) != (b is None):
            raise ValueError(f"{name} and its log probabilities go together")
        width[name] = 0
        if a is not None:
            if a.dim() != 2 or a.shape[0] != N or tuple(b.shape) != tuple(a.shape):
                raise ValueError(f"{name} is {tuple(a.shape)}, its log probabilities {tuple(b.shape)}, "
                                 f"expected [{N}][count] both")
            _typed(a, da, name)
            _typed(b, db, f"log probabilities of {name}")
            _need(a, 0, name)
            _need(b, 0, f"log probabilities of {name}")
            width[name] = int(a.shape[1])
    _typed(entropy, torch.float32, "entropy")
    _need(entropy, N, "entropy")
    _need(workspace, 0, "workspace")
    x = LogprobsArgs()
    _keep(x, (logits, given, given_logp, top_token, top_logp, entropy, workspace))
    x.n_rows, x.vocab, x.top_k, x.n_given = N, V, width["top_token"], width["given"]
    x.in_dtype = GDN_BF16 if logits.dtype == torch.bfloat16 else GDN_F32
    x.logit_stride = int(logits.stride(0)) if N > 1 else max(V, int(logits.shape[1]))
    x.logits, x.given, x.given_logp = _dev(logits), _dev(given), _dev(given_logp)
    x.top_token, x.top_logp, x.entropy = _dev(top_token), _dev(top_logp), _dev(entropy)
    x.workspace = _dev(workspace)
    x.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return x


def token_logprobs(args: LogprobsArgs, stream=None):
    """Log probabilities of the given tokens, the entropy and the top alternatives of every row."""
    _same_device(args, (), "token_logprobs")
    _check(lib().gdn_token_logprobs(ctypes.byref(args), _stream(stream)), "gdn_token_logprobs")
