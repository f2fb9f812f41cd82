"""Python binding of libllama_b200.so: argument marshalling only.

Every step of the forward pass runs in the library's CUDA kernels; PyTorch
supplies device memory (one arena tensor per model) and the current stream.
Importing this package without the built library raises ImportError: there
is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
import re
import traceback

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libllama_b200.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "llama_b200.h")

F32, BF16 = 0, 1
STATUS = {0: "ok", -1: "invalid argument", -2: "arena or workspace too small", -3: "CUDA error",
          -4: "bounded device wait expired", -5: "call out of order"}


class LlamaError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({code})")
        self.code = code


class LlamaConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("ffn_hidden", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("rope_theta", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("max_seq", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("bias", ctypes.c_int32), ("tp_size", ctypes.c_int32), ("tp_rank", ctypes.c_int32),
                ("kv_pages", ctypes.c_int32)]


class LlamaBatchPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "pages_per_seq", "n_pages", "free_capacity", "max_rows", "n_adapters",
                                              "max_tiles")] + \
               [(n, ctypes.c_void_p) for n in ("d_past", "d_new", "d_free", "d_n_free", "d_adapter", "d_table", "d_cu", "d_kv_len",
                                               "d_admitted", "d_n_free_out", "d_slots", "d_pos", "d_seq", "d_lora_rows",
                                               "d_lora_tiles", "d_n_tiles", "d_work")]


# int (*)(float* d_buf, uint64_t count, void* stream, void* ctx): the exchange of a shard
ALLREDUCE_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python decoder_only_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, U64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_float
    I64 = ctypes.c_int64
    sig = {
        "llama_model_bytes": [P, P],
        "llama_init_weights": [P, ctypes.c_uint32, P, U64, P, P],
        "llama_prefill": [P, P, I, I, P, P],
        "llama_prefill_ragged": [P, P, I, I, P, P, P],
        "llama_positions": [P, P, I],
        "llama_prefill_trunk": [P, P, I, I, P, P],
        "llama_decode_step": [P, P, P, P, P],
        "llama_generate": [P, P, I, P, P],
        "llama_position": [P],
        "llama_model_tensor": [P, ctypes.c_char_p, I, P, P],
        "llama_last_error": [P],
        "llama_free": [P],
        "llama_status_str": [ctypes.c_int],
        "llama_op_rmsnorm": [I, P, P, P, I, I, F, P],
        "llama_op_gemm": [I, P, P, P, I, I, I, I, P],
        "llama_op_attention_prefill": [I, P, P, P, P, I, I, I, I, I, P],
        "llama_op_attention_decode": [I, P, P, P, P, I, I, I, I, I, P, U64, P],
        "llama_op_attention_decode_work_bytes": [I, I, I, I],
        "llama_op_attention_decode_noalloc": [I, P, P, P, P, I, I, I, I, I, P],
        "llama_op_argmax": [P, I, I, P, P],
        "llama_op_last_error": [],
        "llama_set_allreduce": [P, ALLREDUCE_FN, P, I],
        "llama_tp_shard": [P, P],
        "llama_set_pages": [P, P, I, I, P],
        "llama_rewind": [P, I, P],
        "llama_complete": [P, P, I, I, P, I, P, P],
        "llama_op_batch_plan": [P, P],
        "llama_kv4_pool_bytes": [I, I, I],
        "llama_op_kv4_append": [I, P, P, P, P, I, I, I, I64, I64, I, P],
        "llama_op_kv4_read": [I, P, P, P, P, I, I, I, I, P],
        "llama_op_attention_kv4": [I, P, I64, P, I, P, I, P, P, I, P, I, I, I, I, I, P, U64, P],
        "llama_op_attention_kv4_work_bytes": [I, I, I, I],
        "llama_op_lora": [I, P, I64, P, P, P, P, I64, P, P, P, I, I, I, I, I, I, P, U64, P],
        "llama_op_lora_work_bytes": [I, I],
        "llama_kernel_launches": [],
        "llama_step_timeline": [P, P, ctypes.c_int64, P, P],
        "llama_debug_gemm_timeout": [P],
        "llama_profile_enable": [I],
        "llama_profile_reset": [],
        "llama_profile_count": [],
        "llama_profile_entry": [I, P, P, P, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.llama_free.restype = None
    lib.llama_profile_reset.restype = None
    lib.llama_kernel_launches.restype = ctypes.c_int64
    lib.llama_status_str.restype = ctypes.c_char_p
    lib.llama_op_attention_decode_work_bytes.restype = U64
    lib.llama_kv4_pool_bytes.restype = U64
    lib.llama_op_attention_kv4_work_bytes.restype = U64
    lib.llama_op_lora_work_bytes.restype = U64
    return lib


lib = _load()


def header_symbols() -> list[str]:
    """Names of the entry points include/llama_b200.h declares."""
    with open(HEADER_PATH) as f:
        return re.findall(r"^LLAMA_API\s+[\w\s\*]+?\b(llama_\w+)\s*\(", f.read(), flags=re.M)


def _check(rc: int, what: str):
    if rc != 0:
        raise LlamaError(rc, what)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def make_config(shape, max_batch: int, max_seq: int, tp=None, kv_pages: int = 0) -> LlamaConfig:
    """`shape`: any object with n_layers, d_model, n_heads, head_dim,
    ffn_hidden, vocab, dtype ('bf16' | 'f32'), norm_eps, rope_theta.
    `tp`: (rank, size) of a tensor-parallel shard, or None.  `kv_pages`:
    pages of 128 positions in a paged KV cache (0: contiguous)."""
    rank, size = tp if tp is not None else (0, 0)
    return LlamaConfig(shape.n_layers, shape.d_model, shape.n_heads, shape.head_dim, shape.ffn_hidden,
                       shape.vocab, shape.norm_eps, shape.rope_theta, BF16 if shape.dtype == "bf16" else F32,
                       max_batch, max_seq, int(getattr(shape, "n_kv_heads", 0) or 0),
                       int(bool(getattr(shape, "bias", False))), size, rank, kv_pages)


def tp_shard(shape, rank: int, size: int) -> dict:
    """The slices shard `rank` of `size` holds (llama_tp_shard)."""
    cfg = make_config(shape, 1, 1, (rank, size))
    out = (ctypes.c_int32 * 6)()
    _check(lib.llama_tp_shard(ctypes.byref(cfg), ctypes.cast(out, ctypes.c_void_p)), "llama_tp_shard")
    return dict(head0=out[0], heads=out[1], kv_head0=out[2], kv_heads=out[3], hidden0=out[4], hidden=out[5])


def allreduce_callback(resolve, reduce):
    """The C exchange (llama_allreduce_fn) around two Python callables:
    resolve(ptr, count) -> the float32 tensor of `count` elements at `ptr`;
    reduce(buf, stream) queues the sum over the shards of `buf` in place on
    `stream` (a torch stream, or None for host tensors).  Exceptions are
    printed and reported to the library as a failed exchange."""
    streams = {}

    def cb(ptr, count, stream, ctx):
        try:
            buf = resolve(ptr or 0, int(count))
            st = None
            if stream:
                st = streams.get(stream)
                if st is None:
                    st = streams[stream] = torch.cuda.ExternalStream(stream)
            reduce(buf, st)
            return 0
        except Exception:
            traceback.print_exc()
            return 1

    return ALLREDUCE_FN(cb)


def dist_allreduce(group=None):
    """reduce(buf, stream) for allreduce_callback / Model.set_allreduce: one
    torch.distributed sum all-reduce (NCCL between GPUs) queued on `stream`."""
    import torch.distributed as dist

    def reduce(buf, stream):
        if stream is None:
            dist.all_reduce(buf, group=group)
        else:
            with torch.cuda.stream(stream):
                dist.all_reduce(buf, group=group)

    return reduce


def model_bytes(cfg: LlamaConfig) -> int:
    n = ctypes.c_uint64()
    _check(lib.llama_model_bytes(ctypes.byref(cfg), ctypes.byref(n)), "llama_model_bytes")
    return n.value


class Model:
    """One model in one device arena.  Weights are generated on the device."""

    def __init__(self, shape, max_batch: int, max_seq: int, seed: int = 0, tp=None, kv_pages: int = 0):
        self.shape = shape
        self.cfg = make_config(shape, max_batch, max_seq, tp, kv_pages)
        nbytes = model_bytes(self.cfg)
        self.arena = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        h = ctypes.c_void_p()
        _check(lib.llama_init_weights(ctypes.byref(self.cfg), seed, _ptr(self.arena), nbytes, _stream(),
                                      ctypes.byref(h)), "llama_init_weights")
        self.h = h
        self.wdtype = torch.bfloat16 if shape.dtype == "bf16" else torch.float32

    def close(self):
        if self.h:
            lib.llama_free(self.h)
            self.h = None

    def set_pages(self, table):
        """Page table of a paged KV cache (llama_set_pages): table[b][p] is the
        pool page of sequence b's positions 128 p .. 128 p + 127."""
        rows = [list(map(int, r)) for r in table]
        B, n = len(rows), len(rows[0])
        flat = (ctypes.c_int32 * (B * n))(*[v for r in rows for v in r])
        _check(lib.llama_set_pages(self.h, ctypes.cast(flat, ctypes.c_void_p), B, n, _stream()), "llama_set_pages")

    def set_allreduce(self, reduce, chunks: int = 4):
        """Installs the exchange of a tensor-parallel shard (llama_set_allreduce):
        reduce(buf, stream) sums `buf`, a float32 view of trunk rows in this
        model's arena, over the shards in place on `stream`."""
        arena = self.arena

        def resolve(ptr, count):
            off = ptr - arena.data_ptr()
            return arena[off:off + 4 * count].view(torch.float32)

        self._allreduce_cb = allreduce_callback(resolve, reduce)   # kept alive with the model
        _check(lib.llama_set_allreduce(self.h, self._allreduce_cb, None, chunks), "llama_set_allreduce")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def position(self) -> int:
        return lib.llama_position(self.h)

    def prefill(self, tokens: torch.Tensor, logits: bool = True, out: torch.Tensor | None = None,
                lens=None):
        """tokens int32 [B, S] on the device -> logits fp32 [B, S, V] (or None).
        With ``lens`` (B ints) the batch is ragged: sequence b is its first
        lens[b] tokens (llama_prefill_ragged)."""
        B, S = tokens.shape
        tokens = tokens.contiguous()
        if logits and out is None:
            out = torch.empty(B, S, self.cfg.vocab, dtype=torch.float32, device="cuda")
        if lens is None:
            _check(lib.llama_prefill(self.h, _ptr(tokens), B, S, _ptr(out if logits else None), _stream()),
                   "llama_prefill")
        else:
            h_lens = (ctypes.c_int32 * B)(*[int(x) for x in lens])
            _check(lib.llama_prefill_ragged(self.h, _ptr(tokens), B, S, ctypes.cast(h_lens, ctypes.c_void_p),
                                            _ptr(out if logits else None), _stream()), "llama_prefill_ragged")
        return out if logits else None

    def positions(self):
        """Each sequence's decode position (host ints)."""
        cap = max(int(self.cfg.max_batch), 1)
        buf = (ctypes.c_int32 * cap)()
        n = lib.llama_positions(self.h, ctypes.cast(buf, ctypes.c_void_p), cap)
        _check(min(n, 0), "llama_positions")
        return [buf[i] for i in range(n)]

    def complete(self, tokens_host: torch.Tensor, n_steps: int, logits: torch.Tensor | None = None,
                 out_host: torch.Tensor | None = None) -> torch.Tensor:
        """Host int32 [B, S] prompt -> host int32 [n_steps, B] greedy tokens
        (llama_complete; pass pinned tensors for asynchronous copies)."""
        B, S = tokens_host.shape
        if out_host is None:
            out_host = torch.empty(n_steps, B, dtype=torch.int32, pin_memory=True)
        _check(lib.llama_complete(self.h, _ptr(tokens_host.contiguous()), B, S, _ptr(logits), n_steps,
                                  _ptr(out_host), _stream()), "llama_complete")
        return out_host

    def rewind(self, position: int):
        _check(lib.llama_rewind(self.h, position, _stream()), "llama_rewind")

    def prefill_trunk(self, x: torch.Tensor, out: torch.Tensor | None = None):
        """x fp32 [B, S, d] -> trunk after the blocks, fp32 [B, S, d]."""
        B, S, _ = x.shape
        x = x.contiguous()
        y = torch.empty_like(x) if out is None else out
        _check(lib.llama_prefill_trunk(self.h, _ptr(x), B, S, _ptr(y), _stream()), "llama_prefill_trunk")
        return y

    def decode_step(self, tokens: torch.Tensor, logits: bool = True):
        B = tokens.shape[0]
        nxt = torch.empty(B, dtype=torch.int32, device="cuda")
        lg = torch.empty(B, self.cfg.vocab, dtype=torch.float32, device="cuda") if logits else None
        _check(lib.llama_decode_step(self.h, _ptr(tokens.contiguous()), _ptr(nxt), _ptr(lg), _stream()),
               "llama_decode_step")
        return nxt, lg

    def generate(self, first: torch.Tensor | None, n_steps: int, out: torch.Tensor | None = None,
                 batch: int | None = None):
        """n_steps greedy tokens [n_steps, B]; first=None continues from the
        prefill's own greedy choice."""
        B = first.shape[0] if first is not None else batch
        out = torch.empty(n_steps, B, dtype=torch.int32, device="cuda") if out is None else out
        f = None if first is None else first.contiguous()
        _check(lib.llama_generate(self.h, _ptr(f), n_steps, _ptr(out), _stream()), "llama_generate")
        return out

    def tensor(self, name: str, layer: int = 0, dtype=None, shape=None) -> torch.Tensor:
        """A view of an internal buffer (see llama_model_tensor)."""
        p, n = ctypes.c_void_p(), ctypes.c_uint64()
        _check(lib.llama_model_tensor(self.h, name.encode(), layer, ctypes.byref(p), ctypes.byref(n)),
               "llama_model_tensor")
        off = p.value - self.arena.data_ptr()
        t = self.arena[off:off + n.value]
        if dtype is not None:
            t = t.view(dtype)
        if shape is not None:
            t = t[: int(torch.Size(shape).numel())].view(shape)
        return t

    def step_timeline(self):
        """[ctas, phases, 2] ns stamps of the last decode step run while
        profiling was enabled (bf16 models)."""
        import numpy as np
        c, p = ctypes.c_int32(), ctypes.c_int32()
        _check(lib.llama_step_timeline(self.h, None, 0, ctypes.byref(c), ctypes.byref(p)), "llama_step_timeline")
        out = np.zeros((c.value, p.value, 2), dtype=np.uint64)
        _check(lib.llama_step_timeline(self.h, ctypes.c_void_p(out.ctypes.data), out.size, None, None),
               "llama_step_timeline")
        return out

    def last_error(self) -> int:
        return lib.llama_last_error(self.h)


# ----------------------------------------------------------------- instrumentation

def kernel_launches() -> int:
    return int(lib.llama_kernel_launches())


def profile_enable(on: bool = True):
    lib.llama_profile_enable(1 if on else 0)


def profile_reset():
    lib.llama_profile_reset()


def profile_read() -> dict:
    """{region: dict(ms, launches, calls, bytes, flops)} (synchronises)."""
    out = {}
    for i in range(lib.llama_profile_count()):
        name = ctypes.c_char_p()
        ms, by, fl = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
        la, ca = ctypes.c_int64(), ctypes.c_int64()
        _check(lib.llama_profile_entry(i, ctypes.byref(name), ctypes.byref(ms), ctypes.byref(la), ctypes.byref(ca),
                                       ctypes.byref(by), ctypes.byref(fl)), "llama_profile_entry")
        out[name.value.decode()] = dict(ms=ms.value, launches=la.value, calls=ca.value, bytes=by.value,
                                        flops=fl.value)
    return out


# ----------------------------------------------------------------- single ops

def rmsnorm(x: torch.Tensor, g: torch.Tensor, eps: float, out_dtype=torch.bfloat16) -> torch.Tensor:
    rows, d = x.shape
    y = torch.empty(rows, d, dtype=out_dtype, device=x.device)
    _check(lib.llama_op_rmsnorm(_dt(y), _ptr(x.contiguous()), _ptr(g.contiguous()), _ptr(y), rows, d, eps,
                                _stream()), "llama_op_rmsnorm")
    return y


def gemm(A: torch.Tensor, W: torch.Tensor, C: torch.Tensor | None = None, accumulate: bool = False):
    """C (+)= A W^T, A [M, K], W [N, K] (same dtype), C fp32 [M, N]."""
    M, K = A.shape
    N = W.shape[0]
    if C is None:
        C = torch.empty(M, N, dtype=torch.float32, device=A.device)
    _check(lib.llama_op_gemm(_dt(A), _ptr(A.contiguous()), _ptr(W.contiguous()), _ptr(C), M, N, K,
                             1 if accumulate else 0, _stream()), "llama_op_gemm")
    return C


def attention_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
    """q [B, H, S, hd]; k, v [B, H, kv_stride, hd] -> o [B*S, H*hd]."""
    B, H, S, hd = q.shape
    kv_stride = k.shape[2]
    o = torch.empty(B * S, H * hd, dtype=q.dtype, device=q.device)
    _check(lib.llama_op_attention_prefill(_dt(q), _ptr(q.contiguous()), _ptr(k.contiguous()), _ptr(v.contiguous()),
                                          _ptr(o), B, H, S, hd, kv_stride, _stream()), "llama_op_attention_prefill")
    return o


def attention_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, length: int,
                     work: torch.Tensor | None = None) -> torch.Tensor:
    """q [B, H*hd]; k, v [B, H, kv_stride, hd]; keys 0..length-1 -> o [B, H*hd]."""
    B, H, kv_stride, hd = k.shape
    nbytes = lib.llama_op_attention_decode_work_bytes(B, H, length, hd)
    if work is None:
        work = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    o = torch.empty(B, H * hd, dtype=q.dtype, device=q.device)
    _check(lib.llama_op_attention_decode(_dt(q), _ptr(q.contiguous()), _ptr(k.contiguous()), _ptr(v.contiguous()),
                                         _ptr(o), B, H, length, hd, kv_stride, _ptr(work), work.numel(),
                                         _stream()), "llama_op_attention_decode")
    return o


def attention_decode_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, length: int) -> torch.Tensor:
    """attention_decode with the workspace in the library's fixed device
    array: no allocation by the library (see the header for the limit)."""
    B, H, kv_stride, hd = k.shape
    o = torch.empty(B, H * hd, dtype=q.dtype, device=q.device)
    _check(lib.llama_op_attention_decode_noalloc(_dt(q), _ptr(q.contiguous()), _ptr(k.contiguous()),
                                                 _ptr(v.contiguous()), _ptr(o), B, H, length, hd, kv_stride,
                                                 _stream()), "llama_op_attention_decode_noalloc")
    return o


def op_last_error() -> int:
    """Reads and clears the single ops' device error word (synchronises the
    current device): 0, -4 when a bounded device wait expired, -1 when a serving
    op met an index (slot, page, length, row, adapter) outside its range."""
    return int(lib.llama_op_last_error())


def argmax(logits: torch.Tensor) -> torch.Tensor:
    rows, n = logits.shape
    out = torch.empty(rows, dtype=torch.int32, device=logits.device)
    _check(lib.llama_op_argmax(_ptr(logits.contiguous()), rows, n, _ptr(out), _stream()), "llama_op_argmax")
    return out


# ----------------------------------------------------------------- serving ops
# A step of many requests: its plan, the 4-bit paged key/value cache and the
# attention over it, and low-rank adapters.  Calls run on the current stream
# of the current device, which has to hold every tensor.

PLAN_PAGE, LORA_TILE = 128, 64


def _need(ok, what: str):
    if not ok:
        raise LlamaError(-1, what)


def _here(what: str, first: torch.Tensor, *others):
    """The raw current stream, once every tensor is known to be on the current device."""
    dev = first.get_device()
    if dev >= 0 and dev == torch._C._cuda_getDevice():
        for t in others:
            if t is not None and t.get_device() != dev:
                break
        else:
            return torch._C._cuda_getCurrentRawStream(dev)
    raise LlamaError(-1, f"{what}: every tensor has to be on the current CUDA device")


def _i32(what: str, *tensors):
    for t in tensors:
        if t is not None and (t.dtype is not torch.int32 or not t.is_contiguous()):
            raise LlamaError(-1, f"{what}: lengths, tables, slots and plans are contiguous int32 tensors")


def _rows_view(t: torch.Tensor, width: int) -> tuple[torch.Tensor, int]:
    """(t, elements between its rows) for a tensor whose rows (all but the first
    dimension) are contiguous and start on 16 bytes; a copy otherwise."""
    if t.data_ptr() % 16 == 0:
        if t.is_contiguous():
            return t, width
        per16, ld = 16 // t.element_size(), t.stride(0)
        if t[0].is_contiguous() and t.shape[0] > 1 and ld >= width and ld % per16 == 0:
            return t, ld
    return t.clone(memory_format=torch.contiguous_format), width


class BatchPlan:
    """The device buffers of a step's plan (llama_op_batch_plan), kept from step
    to step: cu [B + 1], kv_len [B], admitted [B], n_free [1], slots / pos / seq
    [max_rows] and, with adapters, lora_rows [max_rows], lora_tiles
    [max_tiles, 4], n_tiles [1]; int32, on the current device."""

    def __init__(self, batch: int, max_rows: int, n_adapters: int = 0):
        _need(1 <= batch <= 1024 and 1 <= max_rows <= 1 << 30 and 0 <= n_adapters <= 512, "BatchPlan")
        self.batch, self.max_rows, self.n_adapters = batch, max_rows, n_adapters
        self.max_tiles = -(-max_rows // LORA_TILE) + min(batch, n_adapters)
        sizes = dict(lora_tiles=4 * self.max_tiles if n_adapters else 0, lora_rows=max_rows if n_adapters else 0,
                     n_tiles=1 if n_adapters else 0, cu=batch + 1, kv_len=batch, admitted=batch, n_free=1, slots=max_rows,
                     pos=max_rows, seq=max_rows, work=2 + 2 * batch)
        buf = torch.zeros(sum(-(-n // 4) * 4 for n in sizes.values()), dtype=torch.int32, device="cuda")
        at = 0
        for name, n in sizes.items():          # each on a 16-byte boundary
            setattr(self, name, buf[at:at + n])
            at += -(-n // 4) * 4
        self.lora_tiles = self.lora_tiles.view(-1, 4)
        self._args = a = LlamaBatchPlan(B=batch, max_rows=max_rows, n_adapters=n_adapters, max_tiles=self.max_tiles)
        self._ref = ctypes.byref(a)
        a.d_cu, a.d_kv_len, a.d_admitted, a.d_n_free_out = (t.data_ptr() for t in (self.cu, self.kv_len, self.admitted, self.n_free))
        a.d_slots, a.d_pos, a.d_seq, a.d_work = (t.data_ptr() for t in (self.slots, self.pos, self.seq, self.work))
        if n_adapters:
            a.d_lora_rows, a.d_lora_tiles, a.d_n_tiles = (t.data_ptr() for t in (self.lora_rows, self.lora_tiles, self.n_tiles))


def batch_plan(past: torch.Tensor, new: torch.Tensor, table: torch.Tensor, free: torch.Tensor, n_free: torch.Tensor, *,
               n_pages: int, max_rows: int | None = None, adapter: torch.Tensor | None = None, n_adapters: int = 0,
               out: BatchPlan | None = None) -> BatchPlan:
    """Plans a step on the device (llama_op_batch_plan).  past, new [B]; table
    [B, pages_per_seq], updated in place; free [capacity] and n_free [1], the
    stack of free pages.  `out` reuses a plan's buffers (and takes max_rows and
    n_adapters from it); past may then be its kv_len and n_free its n_free (the
    step after)."""
    B = past.numel()
    if out is None:
        _need(max_rows is not None, "batch_plan: max_rows or out")
        _here("batch_plan", past)
        out = BatchPlan(B, max_rows, n_adapters)
    else:
        _need(max_rows in (None, out.max_rows) and n_adapters in (0, out.n_adapters), "batch_plan: out is of another max_rows or n_adapters")
    stream = _here("batch_plan", past, new, table, free, n_free, adapter, out.cu)
    _i32("batch_plan", past, new, table, free, n_free, adapter)
    _need(out.batch == B and new.numel() == B and table.dim() == 2 and table.shape[0] == B and n_free.numel() == 1,
          "batch_plan: past, new, table, out of one batch")
    _need(out.n_adapters == 0 or (adapter is not None and adapter.numel() == B), "batch_plan: adapter")
    a = out._args
    a.pages_per_seq, a.n_pages, a.free_capacity = table.shape[1], n_pages, free.numel()
    a.d_past, a.d_new, a.d_free, a.d_n_free = past.data_ptr(), new.data_ptr(), free.data_ptr(), n_free.data_ptr()
    a.d_table = table.data_ptr()
    a.d_adapter = adapter.data_ptr() if adapter is not None else None
    _check(lib.llama_op_batch_plan(out._ref, stream), "llama_op_batch_plan")
    return out


def kv4_pool(n_pages: int, n_kv: int, head_dim: int) -> torch.Tensor:
    """An empty 4-bit cache: uint8 [n_pages, n_kv, bytes of a page's head]."""
    n = lib.llama_kv4_pool_bytes(n_pages, n_kv, head_dim)
    _need(n > 0, "kv4_pool")
    return torch.zeros(n_pages, n_kv, n // (n_pages * n_kv), dtype=torch.uint8, device="cuda")


_KV4_HEAD_BYTES = {hd: lib.llama_kv4_pool_bytes(1, 1, hd) for hd in (64, 128)}


def _pool_shape(what: str, pool: torch.Tensor, head_dim: int) -> tuple[int, int]:
    shape = pool.shape
    if pool.dtype is not torch.uint8 or len(shape) != 3 or shape[2] != _KV4_HEAD_BYTES.get(head_dim) or not pool.is_contiguous() \
            or shape[0] == 0 or shape[1] == 0:
        raise LlamaError(-1, f"{what}: pool")
    return shape[0], shape[1]


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor) -> None:
    """Stores k, v [rows, n_kv, head_dim] at slots [rows] (negative: left out) of
    the 4-bit cache (llama_op_kv4_append).  k and v may be views of a wider
    projection's rows."""
    _need(k.dim() == 3 and k.shape == v.shape and k.dtype == v.dtype, "kv4_append: k and v of one shape and type")
    rows, n_kv, hd = k.shape
    n_pages, heads = _pool_shape("kv4_append", pool, hd)
    stream = _here("kv4_append", k, v, slots, pool)
    _i32("kv4_append", slots)
    _need(heads == n_kv and slots.numel() == rows, "kv4_append: pool's heads, slots' rows")
    k, ks = _rows_view(k, n_kv * hd)
    v, vs = _rows_view(v, n_kv * hd)
    _check(lib.llama_op_kv4_append(_dt(k), k.data_ptr(), v.data_ptr(), slots.data_ptr(), pool.data_ptr(), rows, n_kv, hd, ks, vs,
                                   n_pages, stream), "llama_op_kv4_append")


def kv4_read(pool: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype=torch.bfloat16) -> tuple[torch.Tensor, torch.Tensor]:
    """The keys and values held at slots [rows]: two [rows, n_kv, head_dim], zeros
    for negative slots (llama_op_kv4_read)."""
    n_pages, n_kv = _pool_shape("kv4_read", pool, head_dim)
    stream = _here("kv4_read", pool, slots)
    _i32("kv4_read", slots)
    rows = slots.numel()
    k, v = torch.empty((2, rows, n_kv, head_dim), dtype=dtype, device=pool.device).unbind()      # one allocation
    _check(lib.llama_op_kv4_read(_dt(k), pool.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr(), rows, n_kv, head_dim,
                                 n_pages, stream), "llama_op_kv4_read")
    return k, v


def attention_kv4_work(H: int, n_kv: int, head_dim: int, max_q: int = 1) -> torch.Tensor:
    """The workspace of attention_kv4: any batch, any lengths; one per call in flight."""
    n = lib.llama_op_attention_kv4_work_bytes(H, n_kv, head_dim, max_q)
    _need(n > 0, "attention_kv4_work")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def attention_kv4(q: torch.Tensor, pool: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor, cu: torch.Tensor | None = None,
                  max_q: int = 1, out: torch.Tensor | None = None, work: torch.Tensor | None = None) -> torch.Tensor:
    """q [rows, H, head_dim] over the 4-bit cache -> o [rows, H * head_dim]
    (llama_op_attention_kv4).  Request b has kv_len[b] positions and the rows
    cu[b] .. cu[b + 1] - 1 (cu None: one row each).  max_q has to be the most rows
    of a request or more: a request with more is left out, which op_last_error
    reports.  Rows of no request are left as they were in `out` (uninitialised
    without it)."""
    _need(q.dim() == 3, "attention_kv4: q")
    rows, H, hd = q.shape
    n_pages, n_kv = _pool_shape("attention_kv4", pool, hd)
    stream = _here("attention_kv4", q, pool, table, kv_len, cu, out, work)
    _i32("attention_kv4", table, kv_len, cu)
    B = kv_len.numel()
    _need(table.dim() == 2 and table.shape[0] == B and (cu is None or cu.numel() == B + 1), "attention_kv4: table, kv_len, cu of one batch")
    if out is None:
        out = q.new_empty((rows, H * hd))
    else:
        _need(out.dtype == q.dtype and out.is_contiguous() and out.numel() == q.numel(), "attention_kv4: out")
    if work is None:
        work = attention_kv4_work(H, n_kv, hd, max_q)
    _need(work.is_contiguous(), "attention_kv4: work")
    q, stride = _rows_view(q, H * hd)
    _check(lib.llama_op_attention_kv4(_dt(q), q.data_ptr(), stride, pool.data_ptr(), n_pages, table.data_ptr(), table.shape[1],
                                      kv_len.data_ptr(), None if cu is None else cu.data_ptr(), max_q, out.data_ptr(), B, rows, H, n_kv,
                                      hd, work.data_ptr(), work.nbytes, stream), "llama_op_attention_kv4")
    return out


def lora_work(max_rows: int, rank: int) -> torch.Tensor:
    """The workspace of lora for up to max_rows rows; one per call in flight."""
    n = lib.llama_op_lora_work_bytes(max_rows, rank)
    _need(n > 0, "lora_work")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def lora(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, y: torch.Tensor, rows: torch.Tensor,
         tiles: torch.Tensor, n_tiles: torch.Tensor, work: torch.Tensor | None = None) -> torch.Tensor:
    """y[r] += scale[a] (x[r] A[a]^T) B[a]^T for the rows of each adapter a
    (llama_op_lora).  x [rows, d], A [adapters, rank, d], B [adapters, n, rank]
    of one type; scale [adapters] and y [rows, n] fp32; rows, tiles, n_tiles:
    a plan's lora_rows, lora_tiles, n_tiles.  y is updated in place."""
    M, d = x.shape
    n_ad, rank, _ = A.shape
    n = B.shape[1]
    _need(A.shape[2] == d and tuple(B.shape) == (n_ad, n, rank) and x.dtype == A.dtype == B.dtype, "lora: x, A, B")
    _need(A.is_contiguous() and B.is_contiguous() and scale.is_contiguous() and (work is None or work.is_contiguous()),
          "lora: contiguous A, B, scale, work")
    _need(scale.dtype == torch.float32 and scale.numel() == n_ad, "lora: scale")
    _need(y.dtype == torch.float32 and tuple(y.shape) == (M, n) and (n <= 1 or y.stride(1) == 1), "lora: y")
    stream = _here("lora", x, A, B, scale, y, rows, tiles, n_tiles, work)
    _i32("lora", rows, tiles, n_tiles)
    _need(rows.numel() == M and tiles.dim() == 2 and tiles.shape[1] == 4 and n_tiles.numel() == 1, "lora: rows, tiles, n_tiles")
    if M == 0:
        return y
    if work is None:
        work = lora_work(M, rank)
    x, ldx = _rows_view(x, d)
    ldy = y.stride(0) if M > 1 else -(-n // 4) * 4
    _check(lib.llama_op_lora(_dt(x), x.data_ptr(), ldx, A.data_ptr(), B.data_ptr(), scale.data_ptr(), y.data_ptr(), ldy,
                             rows.data_ptr(), tiles.data_ptr(), n_tiles.data_ptr(), tiles.shape[0], M, d, n, rank, n_ad,
                             work.data_ptr(), work.nbytes, stream), "llama_op_lora")
    return y
