"""Python binding of the GB300 GDN speculative tree-verify library.

Argument marshalling only: every step runs in the CUDA kernels of
``libgdn_gb300.so`` behind the C ABI declared in ``include/gdn.h``.  The
functions carry the C names and the C argument order.  Tensor arguments may be
torch tensors (their ``data_ptr()`` is passed) or raw device addresses
(ints); ``stream`` may be a ``torch.cuda.Stream``, a raw handle or None (the
current torch stream when torch has initialised CUDA, else the legacy default
stream).

A non-zero host return code raises :class:`GdnError`.  Device-side errors are
written into the caller's ``status`` tensor and are read by the caller.

There is no CPU fallback: importing this package fails if the library has not
been built (``python gated_deltanet_speculative_gdn_gb300/build.py``).
"""
from __future__ import annotations

import ctypes
import os
import sys
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn_gb300.so")

GDN_OK = 0
GDN_ERR_NULL, GDN_ERR_DIMS, GDN_ERR_STRIDE, GDN_ERR_ALIGN = -1, -2, -3, -4
GDN_ERR_ALIAS, GDN_ERR_LAUNCH, GDN_ERR_TMA, GDN_ERR_ARG = -5, -6, -7, -8
GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_PARENT, GDN_DEV_BAD_SLOT = 1, 2, 3
GDN_DEV_DUP_SLOT, GDN_DEV_BAD_ACCEPTED, GDN_DEV_TIMEOUT = 4, 5, 6
GDN_DEV_BAD_WINDOW, GDN_DEV_BAD_PAGE, GDN_DEV_BAD_LEN = 7, 8, 9
GDN_DEV_BAD_AXIS, GDN_DEV_BAD_TOKEN = 10, 11
GDN_DEV_BAD_BIAS, GDN_DEV_BAD_MASK = 12, 13
GDN_BF16, GDN_FP16, GDN_FP32 = 0, 1, 2

EXPORTED_SYMBOLS = ("gdn_conv_tree_step", "gdn_tree_verify", "gdn_chain_verify", "gdn_commit",
                    "gdn_conv_tree_step_compact", "gdn_commit_compact", "gdn_gated_rmsnorm",
                    "gdn_decode_step", "gdn_rope_append", "gdn_paged_attention",
                    "gdn_attention_workspace_bytes", "gdn_kv_commit", "gdn_tree_accept",
                    "gdn_kvq_block_bytes", "gdn_kvq_append", "gdn_paged_attention_kvq",
                    "gdn_attention_kvq_workspace_bytes", "gdn_kvq_read", "gdn_kvq_commit",
                    "gdn_logits_probs", "gdn_token_commit",
                    "gdn_test_stall_next_verify", "gdn_test_stall_next_attention",
                    "gdn_status_str", "gdn_replay_row_floats")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python gated_deltanet_speculative_gdn_gb300/build.py)")

lib = ctypes.CDLL(LIB_PATH)


class GdnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_seqs", "n_nodes", "n_slots", "h_k", "h_v", "d_k", "d_v", "d_conv", "max_seq_nodes")]

    @classmethod
    def make(cls, n_seqs, n_nodes, n_slots, h_k, h_v, d, max_seq_nodes, d_conv=4):
        return cls(n_seqs, n_nodes, n_slots, h_k, h_v, d, d, d_conv, max_seq_nodes)

    @property
    def conv_channels(self) -> int:
        return 2 * self.h_k * self.d_k + self.h_v * self.d_v


class AttnDims(ctypes.Structure):
    """gdn_attn_dims: the attention layers' shapes and the paged cache's layout."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_seqs", "n_tokens", "max_seq_tokens", "h_q", "h_kv", "d_head", "dtype", "n_pages", "page_size",
        "table_width")] + [(n, ctypes.c_int64) for n in ("page_stride", "token_stride", "head_stride")]

    @classmethod
    def make(cls, n_seqs, n_tokens, max_seq_tokens, h_q, h_kv, d_head, dtype, n_pages, page_size, table_width,
             page_stride=None, token_stride=None, head_stride=None):
        """Strides default to a dense cache of [page][token][head][d_head]."""
        head = d_head if head_stride is None else head_stride
        token = h_kv * d_head if token_stride is None else token_stride
        page = page_size * h_kv * d_head if page_stride is None else page_stride
        return cls(n_seqs, n_tokens, max_seq_tokens, h_q, h_kv, d_head, dtype, n_pages, page_size, table_width,
                   page, token, head)

    @classmethod
    def make_kvq(cls, n_seqs, n_tokens, max_seq_tokens, h_q, h_kv, d_head, dtype, n_pages, page_size, table_width,
                 page_stride=None, head_stride=None):
        """Dims of a 4-bit cache: strides in bytes, by default those of a dense one of [page][head][block]."""
        block = page_size * d_head // 16 * 9
        head = block if head_stride is None else head_stride
        page = h_kv * head if page_stride is None else page_stride
        return cls(n_seqs, n_tokens, max_seq_tokens, h_q, h_kv, d_head, dtype, n_pages, page_size, table_width,
                   page, 0, head)


class GdnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code} ({gdn_status_str(code)})")
        self.code = code


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_DP = ctypes.POINTER(GdnDims)

lib.gdn_conv_tree_step.argtypes = [_DP, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P]
lib.gdn_tree_verify.argtypes = [_DP, _P, _P, _I64, _P, _P, _P, ctypes.c_float, _P, _P, _P,
                                _P, _P, _I64, _P, _P]
lib.gdn_chain_verify.argtypes = lib.gdn_tree_verify.argtypes
lib.gdn_commit.argtypes = [_DP, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _P]
lib.gdn_conv_tree_step_compact.argtypes = [_DP, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P]
lib.gdn_commit_compact.argtypes = [_DP, _P, _P, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P]
lib.gdn_gated_rmsnorm.argtypes = [_DP, _P, _P, _I64, _P, ctypes.c_float, ctypes.c_int, _P, _P]
lib.gdn_test_stall_next_verify.argtypes = [ctypes.c_uint64]
lib.gdn_test_stall_next_verify.restype = None
lib.gdn_test_stall_next_attention.argtypes = [ctypes.c_uint64, ctypes.c_int]
lib.gdn_test_stall_next_attention.restype = None
lib.gdn_decode_step.argtypes = [_DP, _P, _I64, _P, _P, _P, _I64, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P,
                                _P]
_AP = ctypes.POINTER(AttnDims)
_INT = ctypes.c_int
lib.gdn_rope_append.argtypes = [_AP, _P, _I64, _P, _I64, _P, _I64, _P, _P, ctypes.c_float, _P, _INT, _P, _P, _INT, _INT,
                                _P, _P, _P, _P, _I64, _P, _P, _P, _P]
lib.gdn_paged_attention.argtypes = [_AP, _P, _I64, _P, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _P, _P]
lib.gdn_attention_workspace_bytes.argtypes = [_AP]
lib.gdn_attention_workspace_bytes.restype = ctypes.c_size_t
lib.gdn_kv_commit.argtypes = [_AP, _INT, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
lib.gdn_tree_accept.argtypes = [_DP, _INT, _P, _I64, _P, _I64, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
_F = ctypes.c_float
lib.gdn_kvq_block_bytes.argtypes = [_AP]
lib.gdn_kvq_block_bytes.restype = ctypes.c_size_t
lib.gdn_kvq_append.argtypes = [_AP, _P, _I64, _P, _I64, _F, _F, _P, _P, _P, _P, _P, _P, _P]
lib.gdn_kvq_read.argtypes = [_AP, _INT, _I64, _P, _P, _F, _F, _P, _P, _P, _P, _P, _I64, _P, _P]
lib.gdn_paged_attention_kvq.argtypes = [_AP, _P, _I64, _P, _P, _F, _F, _P, _P, _P, _P, _F, _P, _P, _I64, _P, _P]
lib.gdn_attention_kvq_workspace_bytes.argtypes = [_AP]
lib.gdn_attention_kvq_workspace_bytes.restype = ctypes.c_size_t
lib.gdn_kvq_commit.argtypes = lib.gdn_kv_commit.argtypes
lib.gdn_logits_probs.argtypes = [_DP, _INT, _INT, _P, _I64, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _INT, _P, _I64, _P,
                                 _INT, _P, _I64, _P, _P]
lib.gdn_token_commit.argtypes = [_DP, _INT, _P, _P, _P, _P, _P, _INT, _P, _I64, _P, _P]
for _f in ("gdn_rope_append", "gdn_paged_attention", "gdn_kv_commit", "gdn_tree_accept", "gdn_kvq_append", "gdn_kvq_read",
           "gdn_paged_attention_kvq", "gdn_kvq_commit", "gdn_logits_probs", "gdn_token_commit"):
    getattr(lib, _f).restype = ctypes.c_int
for _f in ("gdn_conv_tree_step", "gdn_tree_verify", "gdn_chain_verify", "gdn_commit", "gdn_conv_tree_step_compact",
           "gdn_commit_compact", "gdn_gated_rmsnorm", "gdn_decode_step"):
    getattr(lib, _f).restype = ctypes.c_int
lib.gdn_status_str.argtypes = [ctypes.c_int]
lib.gdn_status_str.restype = ctypes.c_char_p
lib.gdn_replay_row_floats.argtypes = [ctypes.c_int, ctypes.c_int]
lib.gdn_replay_row_floats.restype = ctypes.c_size_t


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        # torch can have initialised CUDA only if something has imported it; an initialised CUDA is an
        # available one, and asking for availability again costs more than a launch
        torch = sys.modules.get("torch")
        if torch is not None and torch.cuda.is_initialized():
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object
            return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int, raise_on_error: bool) -> int:
    if rc != GDN_OK and raise_on_error:
        raise GdnError(fn, rc)
    return rc


def gdn_status_str(code: int) -> str:
    return lib.gdn_status_str(int(code)).decode()


def gdn_replay_row_floats(d_k: int, d_v: int) -> int:
    return int(lib.gdn_replay_row_floats(int(d_k), int(d_v)))


def gdn_conv_tree_step(dims: GdnDims, x, x_stride: int, conv_w, conv_hist, parents, node_off,
                       slot_map, xc, win, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_conv_tree_step(ctypes.byref(dims), _ptr(x), int(x_stride), _ptr(conv_w),
                                _ptr(conv_hist), _ptr(parents), _ptr(node_off), _ptr(slot_map),
                                _ptr(xc), _ptr(win), _ptr(status), _stream(stream))
    return _check("gdn_conv_tree_step", rc, raise_on_error)


def gdn_tree_verify(dims: GdnDims, xc, ba, ba_stride: int, dt_bias, A, ssm, q_scale: float,
                    parents, node_off, slot_map, o, replay, replay_stride: int, status,
                    stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_tree_verify(ctypes.byref(dims), _ptr(xc), _ptr(ba), int(ba_stride), _ptr(dt_bias),
                             _ptr(A), _ptr(ssm), float(q_scale), _ptr(parents), _ptr(node_off),
                             _ptr(slot_map), _ptr(o), _ptr(replay), int(replay_stride),
                             _ptr(status), _stream(stream))
    return _check("gdn_tree_verify", rc, raise_on_error)


def gdn_chain_verify(dims: GdnDims, xc, ba, ba_stride: int, dt_bias, A, ssm, q_scale: float,
                     parents, node_off, slot_map, o, replay, replay_stride: int, status,
                     stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_chain_verify(ctypes.byref(dims), _ptr(xc), _ptr(ba), int(ba_stride), _ptr(dt_bias),
                              _ptr(A), _ptr(ssm), float(q_scale), _ptr(parents), _ptr(node_off),
                              _ptr(slot_map), _ptr(o), _ptr(replay), int(replay_stride),
                              _ptr(status), _stream(stream))
    return _check("gdn_chain_verify", rc, raise_on_error)


def gdn_commit(dims: GdnDims, accepted, parents, node_off, slot_map, replay, replay_stride: int,
               win, ssm, conv_hist, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_commit(ctypes.byref(dims), _ptr(accepted), _ptr(parents), _ptr(node_off),
                        _ptr(slot_map), _ptr(replay), int(replay_stride), _ptr(win), _ptr(ssm),
                        _ptr(conv_hist), _ptr(status), _stream(stream))
    return _check("gdn_commit", rc, raise_on_error)


def gdn_conv_tree_step_compact(dims: GdnDims, x, x_stride: int, conv_w, conv_hist, parents, node_off,
                               slot_map, xc, win_ref, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_conv_tree_step_compact(ctypes.byref(dims), _ptr(x), int(x_stride), _ptr(conv_w),
                                        _ptr(conv_hist), _ptr(parents), _ptr(node_off), _ptr(slot_map),
                                        _ptr(xc), _ptr(win_ref), _ptr(status), _stream(stream))
    return _check("gdn_conv_tree_step_compact", rc, raise_on_error)


def gdn_commit_compact(dims: GdnDims, accepted, parents, node_off, slot_map, replay, replay_stride: int,
                       x, x_stride: int, win_ref, ssm, conv_hist, status, stream=None,
                       raise_on_error: bool = True) -> int:
    rc = lib.gdn_commit_compact(ctypes.byref(dims), _ptr(accepted), _ptr(parents), _ptr(node_off),
                                _ptr(slot_map), _ptr(replay), int(replay_stride), _ptr(x), int(x_stride),
                                _ptr(win_ref), _ptr(ssm), _ptr(conv_hist), _ptr(status), _stream(stream))
    return _check("gdn_commit_compact", rc, raise_on_error)


def gdn_gated_rmsnorm(dims: GdnDims, o, z, z_stride: int, norm_w, eps: float, gate_mode: int, y,
                      stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_gated_rmsnorm(ctypes.byref(dims), _ptr(o), _ptr(z), int(z_stride), _ptr(norm_w), float(eps),
                               int(gate_mode), _ptr(y), _stream(stream))
    return _check("gdn_gated_rmsnorm", rc, raise_on_error)


def gdn_decode_step(dims: GdnDims, x, x_stride: int, conv_w, conv_hist, ba, ba_stride: int, dt_bias, A, ssm,
                    q_scale: float, slot_map, xc, o, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_decode_step(ctypes.byref(dims), _ptr(x), int(x_stride), _ptr(conv_w), _ptr(conv_hist), _ptr(ba),
                             int(ba_stride), _ptr(dt_bias), _ptr(A), _ptr(ssm), float(q_scale), _ptr(slot_map),
                             _ptr(xc), _ptr(o), _ptr(status), _stream(stream))
    return _check("gdn_decode_step", rc, raise_on_error)


def gdn_rope_append(dims: AttnDims, q, q_stride: int, k, k_stride: int, v, v_stride: int, q_norm_w, k_norm_w,
                    eps: float, pos, n_axes: int, inv_freq, axis, rot_dim: int, interleaved: int, node_off, ctx_len,
                    page_table, q_out, q_out_stride: int, k_pool, v_pool, status, stream=None,
                    raise_on_error: bool = True) -> int:
    rc = lib.gdn_rope_append(ctypes.byref(dims), _ptr(q), int(q_stride), _ptr(k), int(k_stride), _ptr(v),
                             int(v_stride), _ptr(q_norm_w), _ptr(k_norm_w), float(eps), _ptr(pos), int(n_axes),
                             _ptr(inv_freq), _ptr(axis), int(rot_dim), int(interleaved), _ptr(node_off),
                             _ptr(ctx_len), _ptr(page_table), _ptr(q_out), int(q_out_stride), _ptr(k_pool),
                             _ptr(v_pool), _ptr(status), _stream(stream))
    return _check("gdn_rope_append", rc, raise_on_error)


def gdn_paged_attention(dims: AttnDims, q, q_stride: int, k_pool, v_pool, page_table, ctx_len, node_off, parents,
                        scale: float, o, workspace, workspace_bytes: int, status, stream=None,
                        raise_on_error: bool = True) -> int:
    rc = lib.gdn_paged_attention(ctypes.byref(dims), _ptr(q), int(q_stride), _ptr(k_pool), _ptr(v_pool),
                                 _ptr(page_table), _ptr(ctx_len), _ptr(node_off), _ptr(parents), float(scale),
                                 _ptr(o), _ptr(workspace), int(workspace_bytes), _ptr(status), _stream(stream))
    return _check("gdn_paged_attention", rc, raise_on_error)


def gdn_attention_workspace_bytes(dims: AttnDims) -> int:
    return int(lib.gdn_attention_workspace_bytes(ctypes.byref(dims)))


def gdn_kv_commit(dims: AttnDims, n_layers: int, layer_stride: int, accepted, parents, node_off, ctx_len, page_table,
                  k_pool, v_pool, new_len, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_kv_commit(ctypes.byref(dims), int(n_layers), int(layer_stride), _ptr(accepted), _ptr(parents),
                           _ptr(node_off), _ptr(ctx_len), _ptr(page_table), _ptr(k_pool), _ptr(v_pool),
                           _ptr(new_len), _ptr(status), _stream(stream))
    return _check("gdn_kv_commit", rc, raise_on_error)


def gdn_kvq_block_bytes(dims: AttnDims) -> int:
    return int(lib.gdn_kvq_block_bytes(ctypes.byref(dims)))


def gdn_kvq_append(dims: AttnDims, k, k_stride: int, v, v_stride: int, k_unit: float, v_unit: float, node_off, ctx_len,
                   page_table, k_pool, v_pool, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_kvq_append(ctypes.byref(dims), _ptr(k), int(k_stride), _ptr(v), int(v_stride), float(k_unit), float(v_unit),
                            _ptr(node_off), _ptr(ctx_len), _ptr(page_table), _ptr(k_pool), _ptr(v_pool), _ptr(status),
                            _stream(stream))
    return _check("gdn_kvq_append", rc, raise_on_error)


def gdn_kvq_read(dims: AttnDims, n_layers: int, layer_stride: int, k_pool, v_pool, k_unit: float, v_unit: float, node_off,
                 start, page_table, k, v, row_stride: int, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_kvq_read(ctypes.byref(dims), int(n_layers), int(layer_stride), _ptr(k_pool), _ptr(v_pool), float(k_unit),
                          float(v_unit), _ptr(node_off), _ptr(start), _ptr(page_table), _ptr(k), _ptr(v), int(row_stride),
                          _ptr(status), _stream(stream))
    return _check("gdn_kvq_read", rc, raise_on_error)


def gdn_paged_attention_kvq(dims: AttnDims, q, q_stride: int, k_pool, v_pool, k_unit: float, v_unit: float, page_table, ctx_len,
                            node_off, parents, scale: float, o, workspace, workspace_bytes: int, status, stream=None,
                            raise_on_error: bool = True) -> int:
    rc = lib.gdn_paged_attention_kvq(ctypes.byref(dims), _ptr(q), int(q_stride), _ptr(k_pool), _ptr(v_pool), float(k_unit),
                                     float(v_unit), _ptr(page_table), _ptr(ctx_len), _ptr(node_off), _ptr(parents),
                                     float(scale), _ptr(o), _ptr(workspace), int(workspace_bytes), _ptr(status), _stream(stream))
    return _check("gdn_paged_attention_kvq", rc, raise_on_error)


def gdn_attention_kvq_workspace_bytes(dims: AttnDims) -> int:
    return int(lib.gdn_attention_kvq_workspace_bytes(ctypes.byref(dims)))


def gdn_kvq_commit(dims: AttnDims, n_layers: int, layer_stride: int, accepted, parents, node_off, ctx_len, page_table,
                   k_pool, v_pool, new_len, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_kvq_commit(ctypes.byref(dims), int(n_layers), int(layer_stride), _ptr(accepted), _ptr(parents),
                            _ptr(node_off), _ptr(ctx_len), _ptr(page_table), _ptr(k_pool), _ptr(v_pool), _ptr(new_len),
                            _ptr(status), _stream(stream))
    return _check("gdn_kvq_commit", rc, raise_on_error)


def gdn_logits_probs(dims: GdnDims, vocab: int, dtype: int, logits, logits_stride: int, tokens, parents, node_off, slot_map,
                     history, history_stride: int, repetition, frequency, presence, temperature, bias_off, bias_token,
                     bias_value, n_bias: int, mask, mask_stride: int, mask_row, n_masks: int, p, p_stride: int, status,
                     stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_logits_probs(ctypes.byref(dims), int(vocab), int(dtype), _ptr(logits), int(logits_stride), _ptr(tokens),
                              _ptr(parents), _ptr(node_off), _ptr(slot_map), _ptr(history), int(history_stride),
                              _ptr(repetition), _ptr(frequency), _ptr(presence), _ptr(temperature), _ptr(bias_off),
                              _ptr(bias_token), _ptr(bias_value), int(n_bias), _ptr(mask), int(mask_stride), _ptr(mask_row),
                              int(n_masks), _ptr(p), int(p_stride), _ptr(status), _stream(stream))
    return _check("gdn_logits_probs", rc, raise_on_error)


def gdn_token_commit(dims: GdnDims, vocab: int, tokens, accepted, parents, node_off, slot_map, prompt: int, history,
                     history_stride: int, status, stream=None, raise_on_error: bool = True) -> int:
    rc = lib.gdn_token_commit(ctypes.byref(dims), int(vocab), _ptr(tokens), _ptr(accepted), _ptr(parents), _ptr(node_off),
                              _ptr(slot_map), int(prompt), _ptr(history), int(history_stride), _ptr(status), _stream(stream))
    return _check("gdn_token_commit", rc, raise_on_error)


def gdn_tree_accept(dims: GdnDims, vocab: int, p, p_stride: int, q, q_stride: int, replacement: int, tokens, parents,
                    node_off, u, u_next, accepted, next_token, n_accepted, status, stream=None,
                    raise_on_error: bool = True) -> int:
    rc = lib.gdn_tree_accept(ctypes.byref(dims), int(vocab), _ptr(p), int(p_stride), _ptr(q), int(q_stride),
                             int(replacement), _ptr(tokens), _ptr(parents), _ptr(node_off), _ptr(u), _ptr(u_next),
                             _ptr(accepted), _ptr(next_token), _ptr(n_accepted), _ptr(status), _stream(stream))
    return _check("gdn_tree_accept", rc, raise_on_error)


def gdn_test_stall_next_verify(wait_ns: int) -> None:
    lib.gdn_test_stall_next_verify(int(wait_ns))


def gdn_test_stall_next_attention(wait_ns: int, role: int) -> None:
    lib.gdn_test_stall_next_attention(int(wait_ns), int(role))
