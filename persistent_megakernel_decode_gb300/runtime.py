"""ctypes binding of libmk (argument marshalling only).

Every step of the decode path runs in the library's CUDA kernel; this module
converts Python / torch arguments to the C ABI of ``include/mk.h`` and keeps
the device buffers alive.  There is no CPU fallback: ``load()`` raises when
``libmk.so`` is missing or cannot be loaded.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence

import numpy as np

torch = None  # what works on tensors imports it (need_torch): planning does without

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmk.so")

# ---- constants mirrored from include/mk.h ----
MK_OK, MK_ERR_INVALID, MK_ERR_UNSUPPORTED, MK_ERR_DEADLOCK, MK_ERR_CUDA = 0, 1, 2, 3, 4
MK_ERR_RESIDENCY, MK_ERR_TIMEOUT, MK_ERR_DEVICE_CHECK, MK_ERR_UNBOUND = 5, 6, 7, 8
OP_NAMES = {0: "noop", 1: "counter", 2: "embed", 3: "qkv", 4: "attn", 5: "o", 6: "up", 7: "down", 8: "lm",
            9: "glm_a0", 10: "glm_gemm", 11: "glm_fin", 12: "norm", 13: "attn_pool"}
OPCODE = {v: k for k, v in OP_NAMES.items()}
MODE_MEGAKERNEL, MODE_PER_OP = 0, 1
SCHED_DEFAULT, SCHED_BYTES, SCHED_TIMED = 0, 1, 2
RUN_HOST_TOKENS, RUN_TRACE, RUN_ONE_LAUNCH = 1, 2, 4
PAIR_WHOLE, PAIR_TILE, PAIR_TILE_COVER, PAIR_TILE_REDUCE = 0, 1, 2, 3
TASK_FIELDS = 24
BIND = {n: i for i, n in enumerate([
    "embed", "lm_head", "norm_final", "wq", "wk", "wv", "wo", "wg", "wu", "wd", "norm_attn", "norm_mlp",
    "qnorm", "knorm", "kcache", "vcache", "tokens", "logits", "argmax", "hidden",
    # GLM pre-attention block
    "glm_x", "glm_res", "glm_norm", "glm_res_out", "glm_qa", "glm_sa", "glm_w_qkva", "glm_s_qkva", "glm_w_gate",
    "glm_s_gate", "glm_w_ik", "glm_s_ik", "glm_w_qb", "glm_s_qb", "glm_w_iq", "glm_s_iq", "glm_qkva", "glm_ik",
    "glm_qb", "glm_sb", "glm_gate", "glm_q", "glm_iq", "glm_latent", "glm_index",
    # FP8 projections: block scales of wq .. wd
    "sq", "sk", "sv", "so", "sg", "su", "sd"])}
SCALE_OF = {"wq": "sq", "wk": "sk", "wv": "sv", "wo": "so", "wg": "sg", "wu": "su", "wd": "sd"}
PER_LAYER = ("wq", "wk", "wv", "wo", "wg", "wu", "wd", "norm_attn", "norm_mlp", "qnorm", "knorm")

EXPORTED = ["mk_plan", "mk_plan_graph", "mk_plan_info_get", "mk_plan_export", "mk_bind", "mk_run",
            "mk_sync_status", "mk_read_counters", "mk_read_trace", "mk_free", "mk_last_error", "mk_argmax_index",
            "mk_run_static", "mk_plan_glm", "mk_launch_probe", "mk_plan_export_attn_table",
            "mk_cache_store", "mk_cache_load", "mk_cache_attend", "mk_cache_attend_workspace", "mk_cache_copy",
            "mk_cache_status", "mk_pages_create", "mk_pages_alloc", "mk_pages_share", "mk_pages_release",
            "mk_pages_compact", "mk_pages_info", "mk_pages_free", "mk_sample"]
STATIC_WORKSPACE_BYTES = 64 << 20


class MkError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmk error {code}: {msg}")
        self.code = code


class ModelDesc(C.Structure):
    _fields_ = [("layers", C.c_int), ("hidden", C.c_int), ("q_heads", C.c_int), ("kv_heads", C.c_int),
                ("head_dim", C.c_int), ("ffn", C.c_int), ("vocab", C.c_int), ("qk_norm", C.c_int),
                ("eps", C.c_float), ("rope_theta", C.c_float), ("weight_fp8", C.c_int)]


class StepDesc(C.Structure):
    _fields_ = [("batch", C.c_int), ("seq_len0", C.POINTER(C.c_int)), ("max_steps", C.c_int),
                ("cache_slots", C.c_int), ("capture_hidden", C.c_int)]


class TargetDesc(C.Structure):
    _fields_ = [("num_sms", C.c_int), ("smem_per_cta", C.c_int), ("mode", C.c_int), ("rows_qkv", C.c_int),
                ("rows_o", C.c_int), ("rows_up", C.c_int), ("rows_down", C.c_int), ("kchunk_down", C.c_int),
                ("rows_lm", C.c_int), ("attn_split", C.c_int), ("page_bytes", C.c_int),
                ("schedule", C.c_int), ("tc_tiles", C.c_int), ("attn_pool", C.c_int)]


class GlmDesc(C.Structure):
    _fields_ = [(n, C.c_int) for n in (
        "requests", "tokens", "hidden", "q_lora", "kv_lora", "rope", "q_heads", "q_head_dim", "gate_heads",
        "idx_heads", "idx_dim", "cache_slots", "pos0", "max_steps")] + [("eps", C.c_float), ("rope_theta", C.c_float)]


class PlanInfo(C.Structure):
    _fields_ = [(n, C.c_int) for n in (
        "num_workers", "lmax", "num_tasks", "num_events", "num_ops", "num_launches", "num_pages", "page_bytes",
        "smem_bytes", "act_bytes", "rows_qkv", "rows_o", "rows_up", "rows_down", "kchunk_down", "rows_lm",
        "attn_split", "total_slots")] + [("workspace_bytes", C.c_uint64), ("scratch_offset", C.c_uint64),
                                          ("algorithmic_bytes_step", C.c_uint64)] + [
        (n, C.c_int) for n in ("tc_tiles", "ksplit_qkv", "ksplit_o", "weight_fp8", "attn_table_rows")]


class GraphOp(C.Structure):
    _fields_ = [("grid", C.c_int * 3), ("cost", C.c_int)]


class GraphEdge(C.Structure):
    _fields_ = [("prod", C.c_int), ("cons", C.c_int), ("out_map", C.c_int * 3), ("in_map", C.c_int * 3)]


class GraphPub(C.Structure):
    _fields_ = [("prod", C.c_int), ("first_pub", C.c_int), ("num_pub", C.c_int), ("strategy", C.c_int),
                ("k", C.c_int), ("num_cons", C.c_int), ("cons", C.c_int * 4)]


class GraphDesc(C.Structure):
    _fields_ = [("num_ops", C.c_int), ("ops", C.POINTER(GraphOp)), ("num_edges", C.c_int),
                ("edges", C.POINTER(GraphEdge)), ("num_pubs", C.c_int), ("pubs", C.POINTER(GraphPub)),
                ("round_robin", C.c_int)]


class ErrorRecord(C.Structure):
    _fields_ = [("code", C.c_int32), ("worker", C.c_int32), ("slot", C.c_int32), ("event", C.c_int32),
                ("observed", C.c_uint32), ("needed", C.c_uint32), ("opcode", C.c_int32), ("role", C.c_int32)]


class CacheDesc(C.Structure):
    _fields_ = [(n, C.c_uint64) for n in ("k_codes", "v_codes", "k_scales", "v_scales", "status")] + [
        (n, C.c_int) for n in ("layers", "pages", "kv_heads", "page_tokens", "head_dim")]


class CacheRows(C.Structure):
    _fields_ = [("k", C.c_uint64), ("v", C.c_uint64)] + [
        (f"{n}_stride_{x}", C.c_int64) for n in "kv" for x in ("layer", "seq", "token", "head")] + [
        ("rows", C.c_int), ("row0", C.c_uint64)]


class AttendDesc(C.Structure):
    _fields_ = [(n, C.c_uint64) for n in ("q", "out", "lse")] + [
        (n, C.c_int64) for n in ("q_token_stride", "q_head_stride", "out_token_stride", "out_head_stride")] + [
        (n, C.c_uint64) for n in ("table", "lens", "q_start")] + [
        (n, C.c_int) for n in ("batch", "table_width", "q_heads", "tokens", "max_tokens", "window")] + [
        ("scale", C.c_float), ("num_sms", C.c_int)]


class SampleDesc(C.Structure):
    _fields_ = [("logits", C.c_uint64), ("row_stride", C.c_int64), ("batch", C.c_int), ("vocab", C.c_int),
                ("bf16", C.c_int)] + [(n, C.c_uint64) for n in (
                    "u", "tokens", "logprob", "temperature_rows", "top_k_rows", "top_p_rows", "min_p_rows")] + [
        ("temperature", C.c_float), ("top_k", C.c_int), ("top_p", C.c_float), ("min_p", C.c_float)]


_lib = None


def load():
    """Load libmk.so (built by ``build.build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmk.so not found at {LIB_PATH}; build it with "
                           "`python -m persistent_megakernel_decode_gb300.build`")
    lib = C.CDLL(LIB_PATH)
    P = C.c_void_p
    lib.mk_plan.argtypes = [C.POINTER(ModelDesc), C.POINTER(StepDesc), C.POINTER(TargetDesc), C.POINTER(P)]
    lib.mk_plan_graph.argtypes = [C.POINTER(GraphDesc), C.POINTER(TargetDesc), C.POINTER(P)]
    lib.mk_plan_glm.argtypes = [C.POINTER(GlmDesc), C.POINTER(TargetDesc), C.POINTER(P)]
    lib.mk_plan_info_get.argtypes = [P, C.POINTER(PlanInfo)]
    lib.mk_plan_export.argtypes = [P, P, P, P, P]
    lib.mk_plan_export_attn_table.argtypes = [P, P]
    lib.mk_bind.argtypes = [P, C.c_int, C.c_int, C.c_uint64]
    lib.mk_run.argtypes = [P, P, C.c_size_t, C.c_int, C.c_int, C.c_uint32, C.c_uint64, P]
    lib.mk_run_static.argtypes = [P, C.c_int, C.c_int, C.c_uint32, C.c_uint64, P, C.POINTER(C.c_uint64)]
    lib.mk_sync_status.argtypes = [P, P, P, C.POINTER(ErrorRecord)]
    lib.mk_read_counters.argtypes = [P, P, P]
    lib.mk_read_trace.argtypes = [P, P, P]
    lib.mk_launch_probe.argtypes = [C.c_int, C.c_int, P]
    lib.mk_cache_store.argtypes = lib.mk_cache_load.argtypes = [C.POINTER(CacheDesc), C.POINTER(CacheRows), P, C.c_int,
                                                                P, P, C.c_int, C.c_int, P]
    lib.mk_cache_attend.argtypes = [C.POINTER(CacheDesc), C.c_int, C.POINTER(AttendDesc), P, C.c_uint64, P]
    lib.mk_cache_attend_workspace.argtypes = [C.POINTER(CacheDesc), C.POINTER(AttendDesc), C.POINTER(C.c_uint64)]
    lib.mk_cache_copy.argtypes = [C.POINTER(CacheDesc), P, P, C.c_int, P, C.c_int64, P]
    lib.mk_cache_status.argtypes = [C.POINTER(CacheDesc), C.c_int, P, P]
    lib.mk_pages_create.argtypes = [C.c_int, C.POINTER(P)]
    lib.mk_pages_alloc.argtypes = [P, C.c_int, P]
    lib.mk_pages_share.argtypes = lib.mk_pages_release.argtypes = [P, P, C.c_int]
    lib.mk_pages_compact.argtypes = [P, P, P, P]
    lib.mk_pages_info.argtypes = [P, P, P]
    lib.mk_pages_free.argtypes = [P]
    lib.mk_pages_free.restype = None
    lib.mk_sample.argtypes = [C.POINTER(SampleDesc), P]
    lib.mk_free.argtypes = [P]
    lib.mk_free.restype = None
    lib.mk_last_error.restype = C.c_char_p
    lib.mk_argmax_index.argtypes = [C.c_uint64]
    lib.mk_argmax_index.restype = C.c_int32
    _lib = lib
    return lib


def _check(rc: int):
    if rc != MK_OK:
        raise MkError(rc, load().mk_last_error().decode())


def argmax_index(keys: np.ndarray) -> np.ndarray:
    """Token index of each packed argmax key, decoded by the library's
    ``mk_argmax_index``."""
    k = np.asarray(keys, dtype=np.uint64)
    f = load().mk_argmax_index
    return np.array([f(int(v)) for v in k.reshape(-1)], dtype=np.int64).reshape(k.shape)


def _target(num_sms=0, smem_per_cta=0, mode=MODE_MEGAKERNEL, **knobs) -> TargetDesc:
    t = TargetDesc()
    t.num_sms, t.smem_per_cta, t.mode = num_sms, smem_per_cta, mode
    for k, v in knobs.items():
        setattr(t, k, int(v))
    return t


def launch_probe(num_workers: int, cooperative: bool, stream) -> None:
    """Launch the empty probe kernel (see ``mk_launch_probe``) on a torch stream."""
    _check(load().mk_launch_probe(int(num_workers), int(cooperative), C.c_void_p(stream.cuda_stream)))


def need_torch():
    global torch
    import torch


def c_int(x: int) -> int:
    """``x`` held to the range of a C int (ctypes would pass its low 32 bits)."""
    return x if -2 ** 31 <= x < 2 ** 31 else min(max(x, -2 ** 31), 2 ** 31 - 1)


def check_tensor(name, t, index: int, dtype, shape=None):
    """``t`` must lie on CUDA device ``index`` and have the type and the shape."""
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has type {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def launch(index: int, stream, call, *args):
    """``call(*args, stream handle)`` with CUDA device ``index`` current, on ``stream`` (a torch stream of that device) or
    on the device's current torch stream; raises ``MkError`` on a status."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device_index != index:
        raise ValueError(f"a stream of cuda:{stream.device_index} for tensors of cuda:{index}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = call(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = call(*args, handle)
    if rc != MK_OK:
        raise MkError(rc, load().mk_last_error().decode())


def is_current(index: int, stream) -> bool:
    """Is ``stream`` the current torch stream of CUDA device ``index``?"""
    if stream.device_index != index:
        raise ValueError(f"a stream of cuda:{stream.device_index} for tensors of cuda:{index}")
    return stream.cuda_stream == torch._C._cuda_getCurrentRawStream(index)


def beside(index: int, stream, call, *args):
    """``call(*args)`` with ``stream``, another one than the current, as the current stream: what the call makes and
    copies is in order with its launches.  The arguments' memory stays theirs until ``stream`` is past the call, the
    results' until the caller's current stream is past what it had queued when they were dropped."""
    here = torch.cuda.current_stream(index)
    with torch.cuda.stream(stream):
        got = call(*args)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    for t in got or ():
        t.record_stream(here)
    return got


_SETTINGS = ("temperature", "top_k", "top_p", "min_p")


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, stream=None):
    """Draw one token per row of ``logits`` [B, V] (fp32 or bf16 CUDA tensor, rows V or more apart) with the uniforms ``u``
    [B] (fp32, [0, 1)): temperature, then top-k, top-p, min-p, in this order (``mk_sample`` in ``include/mk.h`` has the
    definitions).  Each setting is None (off; temperature 1), a number, or a CUDA tensor of one value per row (fp32;
    int32 for ``top_k``); a temperature of 0 takes the largest logit.  Returns (tokens int32 [B], logprob fp32 [B]: the
    log probability under the filtered distribution); ``tokens``: an int32 [B] tensor to write into.  Asynchronous on
    ``stream`` (default: the current one), where the tensors must be ready; may be captured into a CUDA graph."""
    if torch is None:
        need_torch()
    index = logits.get_device()
    if index < 0:
        raise ValueError("logits must be a CUDA tensor")
    if stream is not None and not is_current(index, stream):
        return beside(index, stream, sample, logits, u, temperature, top_k, top_p, min_p, tokens)
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits must be fp32 or bf16 [B, V], got {logits.dtype} {tuple(logits.shape)}")
    b, v = logits.shape
    stride, inner = logits.stride()
    if inner != 1 and v > 1:
        raise ValueError("logits must be contiguous along the vocabulary")
    check_tensor("u", u, index, torch.float32, (b,))
    if not u.is_contiguous():
        u = u.contiguous()
    values, rows, keep = [1.0, 0, 1.0, 0.0], [0, 0, 0, 0], [u]
    for i, x in enumerate((temperature, top_k, top_p, min_p)):
        if x is None:
            continue
        if isinstance(x, torch.Tensor):
            check_tensor(_SETTINGS[i], x, index, torch.int32 if i == 1 else torch.float32, (b,))
            if not x.is_contiguous():
                x = x.contiguous()
            keep.append(x)  # alive until the launch is queued
            rows[i] = x.data_ptr()
        else:
            values[i] = c_int(x) if i == 1 else x
    device = logits.device
    if tokens is None:
        tokens = torch.empty((b,), dtype=torch.int32, device=device)
    else:
        check_tensor("tokens", tokens, index, torch.int32, (b,))
        if not tokens.is_contiguous():
            raise ValueError("tokens must be contiguous")
    logprob = torch.empty((b,), dtype=torch.float32, device=device)
    d = SampleDesc(logits.data_ptr(), stride if b > 1 else v, b, v, logits.dtype is torch.bfloat16, u.data_ptr(),
                   tokens.data_ptr(), logprob.data_ptr(), *rows, *values)
    launch(index, None, load().mk_sample, C.byref(d))
    return tokens, logprob


class Plan:
    """A host plan (owns host memory only)."""

    def __init__(self, handle):
        self.h = C.c_void_p(handle)
        self._info = None

    @classmethod
    def llama(cls, shape, batch: int, seq_len0: Sequence[int], max_steps: int, cache_slots: int,
              capture_hidden: bool = False, fp8: bool = False, **target):
        """``fp8``: the seven projections are e4m3 with 128 x 128 block scales."""
        lib = load()
        m = ModelDesc(shape.L, shape.H, shape.Hq, shape.Hkv, shape.D, shape.F, shape.V, int(shape.qk_norm),
                      shape.eps, shape.theta, int(fp8))
        lens = (C.c_int * batch)(*[int(x) for x in seq_len0])
        s = StepDesc(batch, lens, max_steps, cache_slots, int(capture_hidden))
        t = _target(**target)
        out = C.c_void_p()
        _check(lib.mk_plan(C.byref(m), C.byref(s), C.byref(t), C.byref(out)))
        return cls(out.value)

    @classmethod
    def graph(cls, ops: List[dict], edges: List[dict] = (), pubs: List[dict] = (), round_robin=False, **target):
        lib = load()
        o = (GraphOp * len(ops))(*[GraphOp((C.c_int * 3)(*op["grid"]), op.get("cost", 1)) for op in ops])
        e = (GraphEdge * max(1, len(edges)))(*[GraphEdge(x["prod"], x["cons"], (C.c_int * 3)(*x["out_map"]),
                                                         (C.c_int * 3)(*x["in_map"])) for x in edges])
        pb = (GraphPub * max(1, len(pubs)))(*[GraphPub(x["prod"], x.get("first_pub", 0), x["num_pub"], x["strategy"],
                                                       x.get("k", 1), len(x["cons"]),
                                                       (C.c_int * 4)(*(list(x["cons"]) + [0] * 4)[:4]))
                                              for x in pubs])
        g = GraphDesc(len(ops), o, len(edges), e, len(pubs), pb, int(round_robin))
        t = _target(**target)
        out = C.c_void_p()
        _check(lib.mk_plan_graph(C.byref(g), C.byref(t), C.byref(out)))
        return cls(out.value)

    @classmethod
    def glm(cls, dims, max_steps: int = 1, **target):
        """Plan the GLM pre-attention block; ``dims`` has the fields of ``mk_glm_desc``."""
        lib = load()
        d = GlmDesc(dims.R, dims.T, dims.H, dims.qlora, dims.kvlora, dims.rope, dims.q_heads, dims.q_head_dim,
                    dims.gate_heads, dims.idx_heads, dims.idx_dim, dims.slots, dims.pos0, max_steps, dims.eps,
                    dims.theta)
        t = _target(**target)
        out = C.c_void_p()
        _check(lib.mk_plan_glm(C.byref(d), C.byref(t), C.byref(out)))
        return cls(out.value)

    def attn_table(self) -> np.ndarray:
        """attn_pool plans: the attention task table, int32 [rows, 32]."""
        n = self.info()["attn_table_rows"]
        out = np.zeros((max(n, 1), 32), np.int32)
        _check(load().mk_plan_export_attn_table(self.h, C.c_void_p(out.ctypes.data)))
        return out[:n]

    def info(self) -> dict:
        if self._info is None:
            i = PlanInfo()
            _check(load().mk_plan_info_get(self.h, C.byref(i)))
            self._info = {f: getattr(i, f) for f, _ in PlanInfo._fields_}
        return self._info

    def export(self):
        i = self.info()
        W, Lm, E, T = i["num_workers"], i["lmax"], i["num_events"], i["num_tasks"]
        total_words = i["total_slots"] * 32
        q = np.zeros(total_words, np.int32)
        ids = np.zeros(total_words // 32, np.int32)
        th = np.zeros(max(E, 1), np.int32)
        tasks = np.zeros((max(T, 1), TASK_FIELDS), np.int32)
        _check(load().mk_plan_export(self.h, q.ctypes.data, ids.ctypes.data, th.ctypes.data, tasks.ctypes.data))
        if i["num_launches"] == 1:
            q = q.reshape(W, Lm, 32)
            ids = ids.reshape(W, Lm)
        return q, ids, th[:E], tasks[:T]

    def bind(self, name: str, ptr: int, layer: int = 0):
        _check(load().mk_bind(self.h, BIND[name], layer, int(ptr)))

    def free(self):
        if self.h and self.h.value:
            load().mk_free(self.h)
            self.h = C.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Session:
    """Device-resident decode state: weights, KV caches, outputs and the workspace.

    ``weights`` follows ``synth.make_weights`` naming (torch bf16 CUDA tensors;
    with ``weights["fp8"]`` the projections are (e4m3 codes, block scales) pairs);
    ``kcache`` / ``vcache`` are [L, B, Hkv, S_max, D] bf16 CUDA tensors, appended in place.
    """

    def __init__(self, shape, weights: Dict[str, object], kcache, vcache, seq_len0: Sequence[int], max_steps: int,
                 capture_hidden: bool = False, stream=None, **target):
        need_torch()
        self.torch = torch
        self.shape = shape
        self.B = len(seq_len0)
        self.max_steps = max_steps
        self.seq_len0 = list(seq_len0)
        dev = kcache.device
        fp8 = bool(weights.get("fp8", False))
        self.plan = Plan.llama(shape, self.B, seq_len0, max_steps, kcache.shape[3], capture_hidden, fp8=fp8, **target)
        info = self.plan.info()
        self.weights, self.kcache, self.vcache = weights, kcache, vcache
        self.tokens = torch.zeros((max_steps + 1, self.B), dtype=torch.int32, device=dev)
        self.logits = torch.zeros((self.B, shape.V), dtype=torch.float32, device=dev)
        self.argmax = torch.zeros((max_steps, self.B), dtype=torch.int64, device=dev)
        self.hidden = torch.zeros((shape.L, self.B, shape.H), dtype=torch.float32, device=dev) if capture_hidden else None
        self.workspace = torch.zeros(info["workspace_bytes"] + 256, dtype=torch.uint8, device=dev)
        off = (-self.workspace.data_ptr()) % 256
        self.ws_ptr = self.workspace.data_ptr() + off
        self.ws_bytes = info["workspace_bytes"]
        p = self.plan
        for n in ("embed", "lm_head", "norm_final"):
            p.bind(n, weights[n].data_ptr())
        for n in PER_LAYER:
            if n in weights:
                for l, t in enumerate(weights[n]):
                    if isinstance(t, tuple):  # FP8: codes, then their block scales
                        p.bind(n, t[0].data_ptr(), l)
                        p.bind(SCALE_OF[n], t[1].data_ptr(), l)
                    else:
                        p.bind(n, t.data_ptr(), l)
        p.bind("kcache", kcache.data_ptr())
        p.bind("vcache", vcache.data_ptr())
        p.bind("tokens", self.tokens.data_ptr())
        p.bind("logits", self.logits.data_ptr())
        p.bind("argmax", self.argmax.data_ptr())
        if self.hidden is not None:
            p.bind("hidden", self.hidden.data_ptr())
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)

    def run(self, first_step: int, num_steps: int = 1, host_tokens: bool = False, trace: bool = False,
            timeout_ns: int = 0, one_launch: bool = False):
        flags = (RUN_HOST_TOKENS if host_tokens else 0) | (RUN_TRACE if trace else 0) | \
            (RUN_ONE_LAUNCH if one_launch else 0)
        _check(load().mk_run(self.plan.h, C.c_void_p(self.ws_ptr), self.ws_bytes, first_step, num_steps, flags,
                             timeout_ns, C.c_void_p(self.stream.cuda_stream)))

    def sync(self) -> ErrorRecord:
        rec = ErrorRecord()
        rc = load().mk_sync_status(self.plan.h, C.c_void_p(self.ws_ptr), C.c_void_p(self.stream.cuda_stream),
                                   C.byref(rec))
        if rc != MK_OK:
            raise MkError(rc, load().mk_last_error().decode())
        return rec

    def run_static(self, first_step: int, num_steps: int = 1, host_tokens: bool = False, timeout_ns: int = 0) -> int:
        """Run through mk_run_static (library-owned workspace, no device allocation).
        Returns the device address of that workspace, for sync_static()."""
        addr = C.c_uint64(0)
        flags = RUN_HOST_TOKENS if host_tokens else 0
        _check(load().mk_run_static(self.plan.h, first_step, num_steps, flags, timeout_ns,
                                    C.c_void_p(self.stream.cuda_stream), C.byref(addr)))
        return addr.value

    def sync_static(self, addr: int) -> ErrorRecord:
        rec = ErrorRecord()
        rc = load().mk_sync_status(self.plan.h, C.c_void_p(addr), C.c_void_p(self.stream.cuda_stream), C.byref(rec))
        if rc != MK_OK:
            raise MkError(rc, load().mk_last_error().decode())
        return rec

    def sample(self, step: int, u, temperature=None, top_k=None, top_p=None, min_p=None):
        """Sample the tokens that follow ``step`` from its logits (see :func:`sample`; ``u`` [B]) into ``tokens[step +
        1]``, where step ``step + 1`` run with ``host_tokens`` reads them.  Runs on the session's stream: ``u`` and the
        settings must be ready there.  Returns (tokens, logprob), both [B]."""
        if not 0 <= step < self.max_steps:
            raise ValueError(f"step {step} outside the planned {self.max_steps}")
        return sample(self.logits, u, temperature, top_k, top_p, min_p, tokens=self.tokens[step + 1], stream=self.stream)

    def generate(self, first_step: int, num_steps: int, u, temperature=None, top_k=None, top_p=None, min_p=None,
                 timeout_ns: int = 0):
        """Decode ``num_steps`` steps from ``tokens[first_step]`` on, each next token sampled with the settings of
        :func:`sample` and the uniforms ``u[i]`` (fp32 [num_steps, B]) instead of taken by argmax.  Returns the sampled
        tokens int32 [num_steps, B] (a view of ``tokens``) and their log probabilities; asynchronous."""
        if first_step < 0 or num_steps < 0 or first_step + num_steps > self.max_steps:
            raise ValueError(f"steps {first_step} .. {first_step + num_steps - 1} outside the planned {self.max_steps}")
        check_tensor("u", u, self.logits.get_device(), self.torch.float32, (num_steps, self.B))
        logs = []
        for i in range(num_steps):
            self.run(first_step + i, 1, host_tokens=True, timeout_ns=timeout_ns)
            logs.append(self.sample(first_step + i, u[i], temperature, top_k, top_p, min_p)[1])
        with self.torch.cuda.stream(self.stream):
            logprob = self.torch.stack(logs) if logs else u.new_empty((0, self.B))
        logprob.record_stream(self.torch.cuda.current_stream(self.logits.device))  # where the caller reads it
        return self.tokens[first_step + 1: first_step + 1 + num_steps], logprob

    def store_kv(self, cache, table, start, count, max_count: Optional[int] = None):
        """Park K/V in an 8-bit paged cache (``kvcache.Kv8Cache`` with this model's layers, heads and head_dim):
        positions ``start[b]`` .. ``start[b] + count[b] - 1`` of every sequence, all layers, into the pages of ``table``
        (int32 CUDA tensors [B, width], [B], [B]).  Runs on the session's stream: these must be ready there."""
        cache.store(self.kcache.transpose(2, 3), self.vcache.transpose(2, 3), table, start, count, row0=start,
                    max_count=max_count, stream=self.stream)

    def load_kv(self, cache, table, start, count, max_count: Optional[int] = None):
        """The inverse of :meth:`store_kv`, on the same stream: bring those positions back from the 8-bit cache."""
        cache.load(self.kcache.transpose(2, 3), self.vcache.transpose(2, 3), table, start, count, row0=start,
                   max_count=max_count, stream=self.stream)

    def step_tokens(self, step: int) -> np.ndarray:
        """Argmax token of every sequence at ``step`` (after sync)."""
        keys = self.argmax[step].cpu().numpy().view(np.uint64)
        return argmax_index(keys)

    def counters(self) -> np.ndarray:
        out = np.zeros(self.plan.info()["num_events"], np.uint32)
        _check(load().mk_read_counters(self.plan.h, C.c_void_p(self.ws_ptr), out.ctypes.data))
        return out

    def trace(self) -> np.ndarray:
        i = self.plan.info()
        out = np.zeros((i["num_workers"], i["lmax"], 16), np.uint64)
        _check(load().mk_read_trace(self.plan.h, C.c_void_p(self.ws_ptr), out.ctypes.data))
        return out


class GlmSession:
    """Device state of the GLM pre-attention block: inputs and FP8 weights from
    ``synth.make_glm_inputs`` (torch CUDA tensors), every output and
    intermediate, and the workspace."""

    OUTPUTS = ("res_out", "qa", "sa", "qkva", "ik", "qb", "sb", "gate", "q", "iq")

    def __init__(self, dims, inputs: Dict[str, object], max_steps: int = 1, stream=None, **target):
        need_torch()
        self.dims = dims
        dev = inputs["x"].device
        self.plan = Plan.glm(dims, max_steps, **target)
        info = self.plan.info()
        M, H, QL = dims.M, dims.H, dims.qlora
        NQKVA = dims.qlora + dims.kvlora + dims.rope
        bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)
        self.out = dict(res_out=z((M, H), bf), qa=z((M, H), u8), sa=z((M, H // 128), f32), qkva=z((M, NQKVA), bf),
                        ik=z((M, dims.idx_dim), bf), qb=z((M, QL), u8), sb=z((M, QL // 128), f32),
                        gate=z((M, dims.gate_heads), bf), q=z((M, dims.q_heads, dims.q_head_dim), bf),
                        iq=z((M, dims.idx_heads, dims.idx_dim), bf))
        self.inputs = inputs
        self.latent = inputs["latent"]
        self.index = inputs["index"]
        self.workspace = torch.zeros(info["workspace_bytes"] + 256, dtype=torch.uint8, device=dev)
        self.ws_ptr = self.workspace.data_ptr() + (-self.workspace.data_ptr()) % 256
        self.ws_bytes = info["workspace_bytes"]
        p = self.plan
        for n in ("x", "res", "norm", "w_qkva", "s_qkva", "w_gate", "s_gate", "w_ik", "s_ik", "w_qb", "s_qb",
                  "w_iq", "s_iq", "latent", "index"):
            p.bind("glm_" + n, inputs[n].data_ptr())
        for n, t in self.out.items():
            p.bind("glm_" + n, t.data_ptr())
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)

    def run(self, first_step: int = 0, num_steps: int = 1, trace: bool = False, timeout_ns: int = 0,
            one_launch: bool = False):
        flags = (RUN_TRACE if trace else 0) | (RUN_ONE_LAUNCH if one_launch else 0)
        _check(load().mk_run(self.plan.h, C.c_void_p(self.ws_ptr), self.ws_bytes, first_step, num_steps, flags,
                             timeout_ns, C.c_void_p(self.stream.cuda_stream)))

    def sync(self) -> ErrorRecord:
        rec = ErrorRecord()
        rc = load().mk_sync_status(self.plan.h, C.c_void_p(self.ws_ptr), C.c_void_p(self.stream.cuda_stream),
                                   C.byref(rec))
        if rc != MK_OK:
            raise MkError(rc, load().mk_last_error().decode())
        return rec

    def counters(self) -> np.ndarray:
        out = np.zeros(self.plan.info()["num_events"], np.uint32)
        _check(load().mk_read_counters(self.plan.h, C.c_void_p(self.ws_ptr), out.ctypes.data))
        return out

    def trace(self) -> np.ndarray:
        i = self.plan.info()
        out = np.zeros((i["num_workers"], i["lmax"], 16), np.uint64)
        _check(load().mk_read_trace(self.plan.h, C.c_void_p(self.ws_ptr), out.ctypes.data))
        return out


class GraphSession:
    """Workspace for an explicit-graph plan (counter tasks only)."""

    def __init__(self, plan: Plan, device="cuda:0", stream=None):
        need_torch()
        self.plan = plan
        info = plan.info()
        self.workspace = torch.zeros(info["workspace_bytes"] + 256, dtype=torch.uint8, device=device)
        self.ws_ptr = self.workspace.data_ptr() + (-self.workspace.data_ptr()) % 256
        self.ws_bytes = info["workspace_bytes"]
        self.stream = stream if stream is not None else torch.cuda.current_stream(torch.device(device))

    def run(self, first_step: int, num_steps: int = 1, timeout_ns: int = 0):
        _check(load().mk_run(self.plan.h, C.c_void_p(self.ws_ptr), self.ws_bytes, first_step, num_steps, 0,
                             timeout_ns, C.c_void_p(self.stream.cuda_stream)))

    def sync(self) -> ErrorRecord:
        rec = ErrorRecord()
        rc = load().mk_sync_status(self.plan.h, C.c_void_p(self.ws_ptr), C.c_void_p(self.stream.cuda_stream),
                                   C.byref(rec))
        if rc not in (MK_OK, MK_ERR_TIMEOUT, MK_ERR_DEVICE_CHECK):
            raise MkError(rc, load().mk_last_error().decode())
        return rec

    def counters(self) -> np.ndarray:
        out = np.zeros(self.plan.info()["num_events"], np.uint32)
        _check(load().mk_read_counters(self.plan.h, C.c_void_p(self.ws_ptr), out.ctypes.data))
        return out
