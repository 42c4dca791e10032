"""Python binding of libdgt (ctypes): argument marshalling only.

Every step of the decode and the GEMM runs in the HIP library; PyTorch only
provides device memory and the current HIP stream.  Function names follow the
C ABI in include/dgt.h one to one.  There is no CPU fallback: when libdgt.so
is missing or no GPU is present the device entry points raise.
"""

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdgt.so")

DGT_FMT_INT8, DGT_FMT_INT4, DGT_FMT_FP8_E4M3, DGT_FMT_BF16_SPLIT = 1, 2, 3, 4
DGT_FMT_INT4_PAIR = 5
DGT_FMT_BF16_EXP = 6
DGT_FMT_BF16_PAIR = 7
DGT_FMT_BF16_WORD = 8
BF16_FORMATS = (DGT_FMT_BF16_SPLIT, DGT_FMT_BF16_EXP, DGT_FMT_BF16_PAIR, DGT_FMT_BF16_WORD)
STATUS = {0: "DGT_OK", -1: "DGT_E_ARG", -2: "DGT_E_SHAPE", -3: "DGT_E_ALPHABET",
          -4: "DGT_E_BUFSIZE", -5: "DGT_E_FORMAT", -6: "DGT_E_CORRUPT", -7: "DGT_E_HIP",
          -8: "DGT_E_UNSUPPORTED"}
EXPORTS = ["dgt_version", "dgt_status_string", "dgt_compress_bound", "dgt_compress_layer",
           "dgt_layer_info", "dgt_decode_tiles", "dgt_gemm_workspace",
           "dgt_fused_decode_gemm", "dgt_dense_workspace", "dgt_dense_gemm",
           "dgt_noalloc_scratch_bytes", "dgt_fused_decode_gemm_noalloc",
           "dgt_page_plan", "dgt_kv_store", "dgt_tree_attention_workspace", "dgt_tree_attention",
           "dgt_lora_workspace", "dgt_lora_add"]
# element types of the serving operators
DGT_ELT_BF16, DGT_ELT_F16, DGT_ELT_F32 = 1, 2, 3
# bytes at the start of dgt_tree_attention's workspace that are zero before its first use
DGT_TREE_ATTENTION_ZEROED = 9216


class DgtError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s failed: %s (%d)" % (where, STATUS.get(code, "?"), code))
        self.code = code


class dgt_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in
                ("fmt", "n", "k", "tile_n", "tile_k", "lanes", "prob_bits", "flags")]


class dgt_info(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in
                 ("fmt", "n", "k", "tile_n", "tile_k", "lanes", "prob_bits", "alphabet",
                  "tiles", "max_tile_words4", "kmax", "flags")] +
                [(n, ctypes.c_uint64) for n in
                 ("table_off", "index_off", "ktab_off", "streams_off", "raw_off",
                  "total_bytes", "stream_bytes")] +
                [("bits_per_weight", ctypes.c_double)])

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


_lib = None


def lib():
    """Load the in-tree libdgt.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libdgt.so not built: run python -m decode_gemm_tile_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, u32, sz = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_size_t
        L.dgt_version.restype = ctypes.c_int
        L.dgt_status_string.restype = ctypes.c_char_p
        L.dgt_status_string.argtypes = [ctypes.c_int]
        L.dgt_compress_bound.restype = sz
        L.dgt_compress_bound.argtypes = [ctypes.POINTER(dgt_params)]
        L.dgt_compress_layer.restype = ctypes.c_int
        L.dgt_compress_layer.argtypes = [ctypes.POINTER(dgt_params), vp, vp, sz,
                                         ctypes.POINTER(sz)]
        L.dgt_layer_info.restype = ctypes.c_int
        L.dgt_layer_info.argtypes = [vp, sz, ctypes.POINTER(dgt_info)]
        L.dgt_decode_tiles.restype = ctypes.c_int
        L.dgt_decode_tiles.argtypes = [vp, ctypes.POINTER(dgt_info), vp, u32, vp, vp, vp]
        L.dgt_gemm_workspace.restype = sz
        L.dgt_gemm_workspace.argtypes = [ctypes.POINTER(dgt_info), u32]
        L.dgt_fused_decode_gemm.restype = ctypes.c_int
        L.dgt_fused_decode_gemm.argtypes = [vp, ctypes.POINTER(dgt_info), vp, u32, vp,
                                            ctypes.c_float, vp, vp, sz, vp, vp]
        L.dgt_noalloc_scratch_bytes.restype = sz
        L.dgt_noalloc_scratch_bytes.argtypes = []
        L.dgt_fused_decode_gemm_noalloc.restype = ctypes.c_int
        L.dgt_fused_decode_gemm_noalloc.argtypes = [vp, ctypes.POINTER(dgt_info), vp, u32, vp,
                                                    ctypes.c_float, vp, vp, vp]
        L.dgt_dense_workspace.restype = sz
        L.dgt_dense_workspace.argtypes = [u32, u32, u32, u32, u32]
        L.dgt_dense_gemm.restype = ctypes.c_int
        L.dgt_dense_gemm.argtypes = [u32, u32, u32, u32, vp, vp, u32, vp, ctypes.c_float, vp,
                                     vp, sz, vp]
        i64, u64 = ctypes.c_int64, ctypes.c_uint64
        L.dgt_page_plan.restype = ctypes.c_int
        L.dgt_page_plan.argtypes = [vp, vp, u32, vp, u32, vp, vp, u32, u32, u32, u32, vp, u32, vp,
                                    vp, vp, vp, vp, vp]
        L.dgt_kv_store.restype = ctypes.c_int
        L.dgt_kv_store.argtypes = [vp, vp, u32, i64, i64, i64, i64, vp, u32, u32, u32, u32, vp, vp,
                                   u32, u32, vp]
        L.dgt_tree_attention_workspace.restype = sz
        L.dgt_tree_attention_workspace.argtypes = [u32, u32, u32, u32, u32]
        L.dgt_tree_attention.restype = ctypes.c_int
        L.dgt_tree_attention.argtypes = [u32, vp, u64, u64, vp, vp, u32, u32, vp, u32, vp, vp, u32,
                                         u32, u32, u32, u32, vp, u32, ctypes.c_float, vp, u64, u64,
                                         vp, sz, vp]
        L.dgt_lora_workspace.restype = sz
        L.dgt_lora_workspace.argtypes = [u32, u32, u32, u32, u32]
        L.dgt_lora_add.restype = ctypes.c_int
        L.dgt_lora_add.argtypes = [vp, u64, vp, u64, vp, vp, vp, u32, vp, vp, u32, u32, u32, u32,
                                   u32, vp, u64, vp, sz, vp]
        _lib = L
    return _lib


def _check(code: int, where: str):
    if code != 0:
        raise DgtError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# Argument checks made before anything is launched: the C ABI receives raw
# device pointers and cannot tell a tensor's shape, dtype, layout or device.
_TWO_BYTE = ("torch.bfloat16", "torch.int16", "torch.uint16", "torch.float16")


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _check_tensor(t, name, shape, dtypes, device):
    """t must be a contiguous tensor of one of `dtypes` (by name), with
    `shape` (None entries are free), on `device`."""
    _need(t is not None, "%s is required" % name)
    _need(hasattr(t, "data_ptr") and hasattr(t, "is_contiguous"), "%s must be a tensor" % name)
    _need(str(t.dtype) in dtypes, "%s has dtype %s, expected one of %s"
          % (name, t.dtype, ", ".join(dtypes)))
    _need(t.dim() == len(shape) and all(s is None or s == d for s, d in zip(shape, t.shape)),
          "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    _need(t.is_contiguous(), "%s must be contiguous" % name)
    _need(t.device == device, "%s is on %s, expected %s" % (name, t.device, device))


def _check_gpu(device):
    """Checked after every argument's shape and dtype: all of them live on
    `device`, which must be a GPU."""
    _need(device.type == "cuda", "arguments must be in GPU memory (the library has no CPU path)")


def _check_status(status, tiles, device):
    if status is not None:
        _check_tensor(status, "status", (None,), ("torch.int32",), device)
        _need(status.numel() >= tiles, "status holds %d entries, the layer has %d tiles"
              % (status.numel(), tiles))


def _check_scales(fmt, scales, n, k, device):
    if fmt in (DGT_FMT_INT4, DGT_FMT_INT4_PAIR):
        _need(k % 128 == 0, "int4 layers need K divisible by 128 (one scale per 128 columns)")
        _check_tensor(scales, "scales", (n, k // 128), _TWO_BYTE, device)
    else:
        _need(scales is None, "scales are only taken by the int4 formats")


# ----------------------------------------------------------------- host side
def dgt_version() -> int:
    return lib().dgt_version()


def dgt_status_string(code: int) -> str:
    return lib().dgt_status_string(code).decode()


def dgt_compress_bound(fmt, n, k, tile_n, tile_k, lanes, prob_bits=12) -> int:
    p = dgt_params(fmt, n, k, tile_n, tile_k, lanes, prob_bits, 0)
    return lib().dgt_compress_bound(ctypes.byref(p))


def dgt_compress_layer(fmt, w, tile_n, tile_k, lanes, prob_bits=None) -> bytes:
    """Offline encoder.  w: [N, K] numpy array (int8 / uint8 codes, or uint16
    bf16 bit patterns for the bf16 formats).  prob_bits defaults to 12 (16 for
    whole bf16 words)."""
    if prob_bits is None:
        prob_bits = 16 if fmt == DGT_FMT_BF16_WORD else 12
    w = np.ascontiguousarray(w)
    n, k = w.shape
    p = dgt_params(fmt, n, k, tile_n, tile_k, lanes, prob_bits, 0)
    cap = lib().dgt_compress_bound(ctypes.byref(p))
    if cap == 0:
        _check(-2, "dgt_compress_bound")
    out = np.empty(cap, dtype=np.uint8)
    size = ctypes.c_size_t(0)
    _check(lib().dgt_compress_layer(ctypes.byref(p), w.ctypes.data_as(ctypes.c_void_p),
                                    out.ctypes.data_as(ctypes.c_void_p), cap,
                                    ctypes.byref(size)), "dgt_compress_layer")
    return out[: size.value].tobytes()


def dgt_layer_info(blob: bytes) -> dgt_info:
    info = dgt_info()
    buf = np.frombuffer(blob, dtype=np.uint8)
    _check(lib().dgt_layer_info(buf.ctypes.data_as(ctypes.c_void_p), len(blob),
                                ctypes.byref(info)), "dgt_layer_info")
    return info


# --------------------------------------------------------------- device side
class DeviceLayer:
    """A blob resident in HBM plus its parsed header."""

    def __init__(self, blob: bytes, device="cuda"):
        import torch
        self.info = dgt_layer_info(blob)
        host = torch.frombuffer(bytearray(blob), dtype=torch.uint8)
        self.blob = host.to(device)
        if self.blob.data_ptr() % 16:
            raise RuntimeError("device blob is not 16-byte aligned")
        self.nbytes = len(blob)


def dgt_decode_tiles(layer: DeviceLayer, tile_ids=None, out=None, status=None, stream=None):
    """Decode tiles into W layout [N, K] (uint8 codes, or int16 bf16 bits)."""
    import torch
    inf = layer.info
    dev = layer.blob.device
    wide = inf.fmt in BF16_FORMATS
    if out is None:
        out = torch.zeros((inf.n, inf.k), dtype=torch.int16 if wide else torch.uint8, device=dev)
    _check_tensor(out, "out", (inf.n, inf.k), _TWO_BYTE if wide else ("torch.uint8", "torch.int8"),
                  dev)
    _check_status(status, inf.tiles, dev)
    ids = None
    n_ids = 0
    if tile_ids is not None:
        if isinstance(tile_ids, torch.Tensor):
            ids = tile_ids
        else:
            a = np.asarray(tile_ids)
            _need(a.dtype.kind in "iub" or a.size == 0, "tile_ids must be a 1-D integer list")
            ids = torch.from_numpy(a.astype(np.int64).reshape(a.shape))
        _need(ids.dim() == 1 and not ids.is_floating_point(), "tile_ids must be a 1-D integer list")
        if ids.numel():
            lo, hi = int(ids.min()), int(ids.max())
            _need(0 <= lo and hi < inf.tiles, "tile ids must lie in [0, %d); got %d..%d"
                  % (inf.tiles, lo, hi))
        _check_gpu(dev)
        ids = ids.to(dtype=torch.int32, device=dev).contiguous()
        n_ids = ids.numel()
        if n_ids == 0:
            return out
    _check_gpu(dev)
    _check(lib().dgt_decode_tiles(_ptr(layer.blob), ctypes.byref(inf), _ptr(ids), n_ids,
                                  _ptr(out), _ptr(status), _stream(stream)),
           "dgt_decode_tiles")
    return out


def dgt_gemm_workspace(layer: DeviceLayer, m: int) -> int:
    return lib().dgt_gemm_workspace(ctypes.byref(layer.info), m)


def alloc_workspace(nbytes: int, device="cuda"):
    import torch
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def dgt_fused_decode_gemm(layer: DeviceLayer, x, scales=None, w_scale=1.0, y=None, ws=None,
                          status=None, stream=None):
    """Y[m, n] = sum_k X[m, k] W[n, k] with W decoded on chip; x: bf16 [M, K]."""
    import torch
    inf = layer.info
    dev = layer.blob.device
    _check_tensor(x, "x", (None, inf.k), ("torch.bfloat16",), dev)
    m = x.shape[0]
    _need(1 <= m, "x needs at least one row")
    if y is None:
        y = torch.empty((m, inf.n), dtype=torch.float32, device=dev)
    _check_tensor(y, "y", (m, inf.n), ("torch.float32",), dev)
    _check_scales(inf.fmt, scales, inf.n, inf.k, dev)
    _check_status(status, inf.tiles, dev)
    if ws is not None:
        _check_tensor(ws, "ws", (None,), ("torch.uint8",), dev)
    _check_gpu(dev)
    if ws is None:
        ws = alloc_workspace(dgt_gemm_workspace(layer, m), dev)
    _check(lib().dgt_fused_decode_gemm(_ptr(layer.blob), ctypes.byref(inf), _ptr(x), m,
                                       _ptr(scales), float(w_scale), _ptr(y), _ptr(ws),
                                       ws.numel(), _ptr(status), _stream(stream)),
           "dgt_fused_decode_gemm")
    return y


def dgt_noalloc_scratch_bytes() -> int:
    return lib().dgt_noalloc_scratch_bytes()


def dgt_fused_decode_gemm_noalloc(layer: DeviceLayer, x, y, scales=None, w_scale=1.0,
                                  status=None, stream=None):
    """dgt_fused_decode_gemm on the library's static scratch: no workspace and,
    given y, no allocation at all."""
    inf = layer.info
    dev = layer.blob.device
    _check_tensor(x, "x", (None, inf.k), ("torch.bfloat16",), dev)
    m = x.shape[0]
    _need(1 <= m, "x needs at least one row")
    _check_tensor(y, "y", (m, inf.n), ("torch.float32",), dev)
    _check_scales(inf.fmt, scales, inf.n, inf.k, dev)
    _check_status(status, inf.tiles, dev)
    _check_gpu(dev)
    _check(lib().dgt_fused_decode_gemm_noalloc(_ptr(layer.blob), ctypes.byref(inf), _ptr(x), m,
                                               _ptr(scales), float(w_scale), _ptr(y),
                                               _ptr(status), _stream(stream)),
           "dgt_fused_decode_gemm_noalloc")
    return y


def dgt_dense_workspace(fmt, n, k, tile_n, m) -> int:
    return lib().dgt_dense_workspace(fmt, n, k, tile_n, m)


def dgt_dense_gemm(fmt, w, x, tile_n=128, scales=None, w_scale=1.0, y=None, ws=None,
                   stream=None):
    """Uncompressed baseline; w: device [N, K] (uint8 codes or bf16 bits)."""
    import torch
    wide = fmt in BF16_FORMATS
    _need(hasattr(w, "shape") and w.dim() == 2, "w must be a 2-D tensor [N, K]")
    n, k = w.shape
    dev = w.device
    _check_tensor(w, "w", (n, k), _TWO_BYTE if wide else ("torch.uint8", "torch.int8"), dev)
    _check_tensor(x, "x", (None, k), ("torch.bfloat16",), dev)
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    _check_tensor(y, "y", (m, n), ("torch.float32",), dev)
    _check_scales(fmt, scales, n, k, dev)
    if ws is not None:
        _check_tensor(ws, "ws", (None,), ("torch.uint8",), dev)
    _check_gpu(dev)
    if ws is None:
        ws = alloc_workspace(dgt_dense_workspace(fmt, n, k, tile_n, m), dev)
    _check(lib().dgt_dense_gemm(fmt, n, k, tile_n, _ptr(w), _ptr(x), m, _ptr(scales),
                                float(w_scale), _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream)), "dgt_dense_gemm")
    return y


# --------------------------------------------------------- serving operators
# Their smallest calls take a few microseconds on the GPU, and what the host does
# before the launch is the larger part of them.  So each function first tests
# everything in one expression; only where that fails are the checks made one by one,
# to say which argument is wrong and how.
def _check_array(t, name, dtype, shape, device):
    """t must be a contiguous tensor of `dtype` and exactly `shape` on `device`."""
    _check_tensor(t, name, shape, (str(dtype),), device)


def _check_rows(t, name, dtypes, shape, device):
    """t must be a tensor of one of `dtypes` and exactly `shape` on `device` whose last
    dimension is contiguous; the other strides are free."""
    _need(t is not None, "%s is required" % name)
    _need(hasattr(t, "data_ptr"), "%s must be a tensor" % name)
    _need(t.dtype in dtypes, "%s has dtype %s, expected one of %s"
          % (name, t.dtype, ", ".join(str(d) for d in dtypes)))
    _need(t.shape == shape, "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    _need(t.stride(-1) == 1 or shape[-1] <= 1, "%s must be contiguous in its last dimension" % name)
    _need(t.device == device, "%s is on %s, expected %s" % (name, t.device, device))


def _dims(t, name, count):
    _need(hasattr(t, "data_ptr") and t.dim() == count, "%s must be a %d-D tensor" % (name, count))
    return t.shape


def _made_on(stream, make):
    """Tensors made inside a call belong to the stream the call runs on, so their memory
    is not handed on while that stream still uses it."""
    import torch
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _call(name, device, stream, *args):
    """One library call on `stream` (default: the device's current stream), with
    `device` as the current device."""
    import torch
    index = device.index
    if stream is not None:
        handle = stream.cuda_stream
    else:  # the current stream's handle, without an object around it
        handle = torch._C._cuda_getCurrentRawStream(index)
    fn = getattr(_lib or lib(), name)
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            code = fn(*args, handle)
    else:
        code = fn(*args, handle)
    if code:
        raise DgtError(code, name)


class PagePlan:
    """What dgt_page_plan returns, on the device: cu int32[requests + 1], slots and
    positions int32[tokens], counts int32[3] (rows needed, the free list's new head,
    requests refused) and, for trees, mask int64[tokens, mask_words] (else None)."""

    __slots__ = ("cu", "slots", "positions", "counts", "mask")

    def __init__(self, cu, slots, positions, counts, mask=None):
        self.cu, self.slots, self.positions, self.counts, self.mask = cu, slots, positions, counts, mask

    @classmethod
    def empty(cls, requests, tokens, mask_words=0, device="cuda"):
        import torch
        def i32(n):
            return torch.empty(n, dtype=torch.int32, device=device)
        mask = torch.empty((tokens, mask_words), dtype=torch.int64, device=device) if mask_words else None
        return cls(i32(requests + 1), i32(tokens), i32(tokens), i32(3), mask)


def _check_page_plan(ctx_lens, new_lens, free_blocks, free_head, block_table, tokens, parents, words, out):
    import torch
    i32, dev = torch.int32, ctx_lens.device
    (requests,) = _dims(ctx_lens, "ctx_lens", 1)
    (free,) = _dims(free_blocks, "free_blocks", 1)
    width = _dims(block_table, "block_table", 2)[1]
    _check_array(ctx_lens, "ctx_lens", i32, (requests,), dev)
    _check_array(new_lens, "new_lens", i32, (requests,), dev)
    _check_array(free_blocks, "free_blocks", i32, (free,), dev)
    _check_array(free_head, "free_head", i32, (1,), dev)
    _check_array(block_table, "block_table", i32, (requests, width), dev)
    _need(tokens >= 0 and words >= 0, "tokens and mask_words must not be negative")
    if parents is not None:
        _check_array(parents, "parents", i32, (tokens,), dev)
    else:
        _need(words == 0, "mask_words needs parents")
    if out is not None:
        _check_array(out.cu, "out.cu", i32, (requests + 1,), dev)
        _check_array(out.slots, "out.slots", i32, (tokens,), dev)
        _check_array(out.positions, "out.positions", i32, (tokens,), dev)
        _check_array(out.counts, "out.counts", i32, (3,), dev)
        if words:
            _check_array(out.mask, "out.mask", torch.int64, (tokens, words), dev)
    _check_gpu(dev)


def dgt_page_plan(ctx_lens, new_lens, free_blocks, free_head, block_table, block_size, num_blocks,
                  tokens, parents=None, mask_words=0, out=None, stream=None):
    """Offsets, slots, positions and tree masks of one step, and the pages it takes from
    the free list (written into block_table).  parents: int32[tokens] for drafted trees,
    with mask_words 64-bit words a token (default: one); None for chains.  out: a PagePlan
    to write into.  out.counts[1:2] is the next step's free_head, also where that step
    writes into the same `out`."""
    import torch
    i32, words = torch.int32, mask_words
    if parents is not None and words == 0:
        words = 1
    _need(hasattr(ctx_lens, "data_ptr"), "ctx_lens must be a 1-D tensor")
    dev, shape = ctx_lens.device, ctx_lens.shape
    try:
        good = (dev.type == "cuda" and ctx_lens.dtype is i32 and ctx_lens.is_contiguous() and len(shape) == 1
                and new_lens.dtype is i32 and new_lens.shape == shape and new_lens.is_contiguous()
                and new_lens.device == dev
                and free_blocks.dtype is i32 and free_blocks.dim() == 1 and free_blocks.is_contiguous()
                and free_blocks.device == dev
                and free_head.dtype is i32 and free_head.shape == (1,) and free_head.device == dev
                and block_table.dtype is i32 and block_table.dim() == 2 and block_table.shape[0] == shape[0]
                and block_table.is_contiguous() and block_table.device == dev and tokens >= 0
                and (words == 0 if parents is None else words > 0 and parents.dtype is i32
                     and parents.shape == (tokens,) and parents.is_contiguous() and parents.device == dev))
        if good and out is not None:
            cu, slots, positions, counts, mask = out.cu, out.slots, out.positions, out.counts, out.mask
            good = (cu.dtype is i32 and cu.shape == (shape[0] + 1,) and cu.is_contiguous() and cu.device == dev
                    and slots.dtype is i32 and slots.shape == (tokens,) and slots.is_contiguous()
                    and slots.device == dev
                    and positions.dtype is i32 and positions.shape == (tokens,) and positions.is_contiguous()
                    and positions.device == dev
                    and counts.dtype is i32 and counts.shape == (3,) and counts.is_contiguous()
                    and counts.device == dev
                    and (words == 0 or mask.dtype is torch.int64 and mask.shape == (tokens, words)
                         and mask.is_contiguous() and mask.device == dev))
    except AttributeError:
        good = False
    if not good:
        _check_page_plan(ctx_lens, new_lens, free_blocks, free_head, block_table, tokens, parents, words, out)
    if out is None:
        out = _made_on(stream, lambda: PagePlan.empty(shape[0], tokens, words, dev))
    # (a step of no tokens still has parents, if only by name)
    up = None if parents is None else parents.data_ptr() or out.counts.data_ptr()
    _call("dgt_page_plan", dev, stream, ctx_lens.data_ptr(), new_lens.data_ptr(), shape[0],
          free_blocks.data_ptr(), free_blocks.shape[0], free_head.data_ptr(), block_table.data_ptr(),
          block_table.shape[1], block_size, num_blocks, tokens, up, words, out.cu.data_ptr(),
          out.slots.data_ptr(), out.positions.data_ptr(), out.mask.data_ptr() if words else None,
          out.counts.data_ptr())
    return out


_ELEMENTS = {}


def _elements():
    """The library's number of each torch dtype that the operators take."""
    if not _ELEMENTS:
        import torch
        _ELEMENTS.update({torch.bfloat16: DGT_ELT_BF16, torch.float16: DGT_ELT_F16, torch.float32: DGT_ELT_F32})
    return _ELEMENTS


def _check_caches(k_cache, v_cache):
    """Shape (blocks, heads, block, dim) of the key pages; the value pages are the same,
    transposed."""
    import torch
    blocks, heads, block, dim = _dims(k_cache, "k_cache", 4)
    dtype = k_cache.dtype
    _need(dtype is torch.bfloat16 or dtype is torch.float16,
          "k_cache has dtype %s, expected torch.bfloat16 or torch.float16" % dtype)
    _check_array(k_cache, "k_cache", dtype, (blocks, heads, block, dim), k_cache.device)
    _check_array(v_cache, "v_cache", dtype, (blocks, heads, dim, block), k_cache.device)
    return blocks, heads, block, dim


def _check_kv_store(k, v, slots, k_cache, v_cache):
    import torch
    blocks, heads, block, dim = _check_caches(k_cache, v_cache)
    dev = k_cache.device
    tokens = _dims(k, "k", 3)[0]
    _check_rows(k, "k", (torch.float32, k_cache.dtype), (tokens, heads, dim), dev)
    _check_rows(v, "v", (k.dtype,), (tokens, heads, dim), dev)
    _check_array(slots, "slots", torch.int32, (tokens,), dev)
    _check_gpu(dev)


def dgt_kv_store(k, v, slots, k_cache, v_cache, stream=None):
    """Write k, v [tokens, heads, dim] (the caches' dtype or float32, any row and head
    strides) into the pages at `slots`; slots outside the pool are skipped."""
    import torch
    elements = _elements()
    try:
        dev, dtype, source = k_cache.device, k_cache.dtype, k.dtype
        blocks, heads, block, dim = k_cache.shape
        tokens = k.shape[0]
        (k_row, k_head, k_one), (v_row, v_head, v_one) = k.stride(), v.stride()
        good = (dev.type == "cuda" and (dtype is torch.bfloat16 or dtype is torch.float16)
                and k_cache.is_contiguous() and v_cache.dtype is dtype
                and v_cache.shape == (blocks, heads, dim, block) and v_cache.is_contiguous()
                and v_cache.device == dev and (source is dtype or source is torch.float32)
                and k.shape == (tokens, heads, dim) and k.device == dev and k_one == 1
                and v.dtype is source and v.shape == (tokens, heads, dim) and v.device == dev and v_one == 1
                and slots.dtype is torch.int32 and slots.shape == (tokens,) and slots.is_contiguous()
                and slots.device == dev)
    except (AttributeError, ValueError, IndexError):
        good = False
    if not good:
        _check_kv_store(k, v, slots, k_cache, v_cache)
    _call("dgt_kv_store", dev, stream, k.data_ptr(), v.data_ptr(), elements[source], k_row, k_head, v_row,
          v_head, slots.data_ptr(), tokens, heads, dim, elements[dtype], k_cache.data_ptr(),
          v_cache.data_ptr(), blocks, block)


def dgt_tree_attention_workspace(q_shape, kv_heads, requests) -> int:
    """Bytes of workspace for queries of shape [tokens, heads, dim]."""
    tokens, heads, dim = q_shape
    n = lib().dgt_tree_attention_workspace(tokens, heads, kv_heads, dim, requests)
    if n == 0:
        raise DgtError(-2, "dgt_tree_attention_workspace")
    return n


def _check_tree_attention(q, k_cache, v_cache, block_table, ctx_lens, cu, mask, out, ws):
    import torch
    blocks, kv_heads, block, dim = _check_caches(k_cache, v_cache)
    dev = k_cache.device
    tokens, heads, _ = _dims(q, "q", 3)
    requests, width = _dims(block_table, "block_table", 2)
    _check_rows(q, "q", (k_cache.dtype,), (tokens, heads, dim), dev)
    _need(heads % max(kv_heads, 1) == 0, "q has %d heads, not a multiple of the cache's %d" % (heads, kv_heads))
    _check_array(block_table, "block_table", torch.int32, (requests, width), dev)
    _check_array(ctx_lens, "ctx_lens", torch.int32, (requests,), dev)
    _check_array(cu, "cu", torch.int32, (requests + 1,), dev)
    if mask is not None:
        words = _dims(mask, "mask", 2)[1]
        _need(words > 0, "mask needs at least one word a token")
        _check_array(mask, "mask", torch.int64, (tokens, words), dev)
    if out is not None:
        _check_rows(out, "out", (q.dtype,), (tokens, heads, dim), dev)
    if ws is not None:
        _check_array(ws, "ws", torch.uint8, (None,), dev)
    _check_gpu(dev)


def _attention_workspace(nbytes, device):
    """A workspace for one call: megabytes of parts, of which only the counters in front are
    cleared."""
    import torch
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws.narrow(0, 0, DGT_TREE_ATTENTION_ZEROED).zero_()
    return ws


def dgt_tree_attention(q, k_cache, v_cache, block_table, ctx_lens, cu, mask=None, scale=None,
                       out=None, ws=None, stream=None):
    """Attention of the new tokens q [tokens, heads, dim] over each request's cached tokens
    and over those of its new tokens (already stored) that `mask` (dgt_page_plan) lets a
    token see; without a mask each sees the ones before it and itself.  scale defaults to
    dim ** -0.5.  Rows past cu[-1] of `out` are not written.  ws: a workspace to keep between
    calls (alloc_workspace); without one each call makes its own."""
    import torch
    i32, words = torch.int32, 0
    try:
        dev, dtype = k_cache.device, k_cache.dtype
        blocks, kv_heads, block, dim = k_cache.shape
        shape = tokens, heads, _ = q.shape
        requests, width = block_table.shape
        q_row, q_head, q_one = q.stride()
        good = (dev.type == "cuda" and (dtype is torch.bfloat16 or dtype is torch.float16)
                and k_cache.is_contiguous() and v_cache.dtype is dtype
                and v_cache.shape == (blocks, kv_heads, dim, block) and v_cache.is_contiguous()
                and v_cache.device == dev
                and q.dtype is dtype and shape[2] == dim and q_one == 1 and q.device == dev
                and kv_heads > 0 and heads % kv_heads == 0
                and block_table.dtype is i32 and block_table.is_contiguous() and block_table.device == dev
                and ctx_lens.dtype is i32 and ctx_lens.shape == (requests,) and ctx_lens.is_contiguous()
                and ctx_lens.device == dev
                and cu.dtype is i32 and cu.shape == (requests + 1,) and cu.is_contiguous() and cu.device == dev)
        if mask is not None:
            words = mask.shape[1]
            good = (good and words > 0 and mask.dtype is torch.int64 and mask.shape == (tokens, words)
                    and mask.is_contiguous() and mask.device == dev)
        if out is not None:
            good = good and out.dtype is dtype and out.shape == shape and out.stride(2) == 1 and out.device == dev
        if ws is not None:
            good = good and ws.dtype is torch.uint8 and ws.dim() == 1 and ws.is_contiguous() and ws.device == dev
    except (AttributeError, ValueError, IndexError):
        good = False
    if not good:
        _check_tree_attention(q, k_cache, v_cache, block_table, ctx_lens, cu, mask, out, ws)
    if out is None:
        out = _made_on(stream, lambda: torch.empty(shape, dtype=dtype, device=dev))
        out_row, out_head = heads * dim, dim
    else:
        out_row, out_head, _ = out.stride()
    if ws is None:
        nbytes = dgt_tree_attention_workspace(shape, kv_heads, requests)
        ws = _made_on(stream, lambda: _attention_workspace(nbytes, dev))
    _call("dgt_tree_attention", dev, stream, _elements()[dtype], q.data_ptr(), q_row, q_head,
          k_cache.data_ptr(), v_cache.data_ptr(), blocks, block, block_table.data_ptr(), width,
          ctx_lens.data_ptr(), cu.data_ptr(), requests, tokens, heads, kv_heads, dim,
          mask.data_ptr() if words and tokens else None, words if tokens else 0,
          dim ** -0.5 if scale is None else scale, out.data_ptr(), out_row, out_head,
          ws.data_ptr(), ws.numel())
    return out


def dgt_lora_workspace(tokens, requests, n, k, rank) -> int:
    nbytes = lib().dgt_lora_workspace(tokens, requests, n, k, rank)
    if nbytes == 0:
        raise DgtError(-2, "dgt_lora_workspace")
    return nbytes


def _check_lora_add(y, x, a, b, scaling, adapters, cu, out, ws):
    import torch
    f32, bf16 = torch.float32, torch.bfloat16
    tokens, n = _dims(y, "y", 2)
    dev = y.device
    k = _dims(x, "x", 2)[1]
    count, rank, _ = _dims(a, "a", 3)
    (requests,) = _dims(adapters, "adapters", 1)
    _check_rows(y, "y", (f32,), (tokens, n), dev)
    _check_rows(x, "x", (bf16,), (tokens, k), dev)
    _check_array(a, "a", bf16, (count, rank, k), dev)
    _check_array(b, "b", bf16, (count, n, rank), dev)
    _check_array(scaling, "scaling", f32, (count,), dev)
    _check_array(adapters, "adapters", torch.int32, (requests,), dev)
    _check_array(cu, "cu", torch.int32, (requests + 1,), dev)
    if out is not None:
        _check_rows(out, "out", (f32,), (tokens, n), dev)
    if ws is not None:
        _check_array(ws, "ws", torch.uint8, (None,), dev)
    _check_gpu(dev)


def dgt_lora_add(y, x, a, b, scaling, adapters, cu, out=None, ws=None, stream=None):
    """out[t] = y[t] + scaling[i] * (x[t] a[i]^T) b[i]^T, i = adapters[request of t] (rows of
    requests with an id outside the adapters: out[t] = y[t]).  x bf16 [tokens, k],
    a bf16 [count, rank, k], b bf16 [count, n, rank], y float32 [tokens, n].  out defaults
    to y (in place)."""
    import torch
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    try:
        dev = y.device
        shape = tokens, n = y.shape
        k = x.shape[1]
        count, rank, _ = a.shape
        (requests,) = adapters.shape
        (y_row, y_one), (x_row, x_one) = y.stride(), x.stride()
        good = (dev.type == "cuda" and y.dtype is f32 and (y_one == 1 or n == 1)
                and x.dtype is bf16 and x.shape == (tokens, k) and x_one == 1 and x.device == dev
                and a.dtype is bf16 and a.shape == (count, rank, k) and a.is_contiguous() and a.device == dev
                and b.dtype is bf16 and b.shape == (count, n, rank) and b.is_contiguous() and b.device == dev
                and scaling.dtype is f32 and scaling.shape == (count,) and scaling.is_contiguous()
                and scaling.device == dev
                and adapters.dtype is i32 and adapters.is_contiguous() and adapters.device == dev
                and cu.dtype is i32 and cu.shape == (requests + 1,) and cu.is_contiguous() and cu.device == dev)
        if out is not None:
            good = (good and out.dtype is f32 and out.shape == shape and (out.stride(1) == 1 or n == 1)
                    and out.device == dev)
        if ws is not None:
            good = good and ws.dtype is torch.uint8 and ws.dim() == 1 and ws.is_contiguous() and ws.device == dev
    except (AttributeError, ValueError, IndexError):
        good = False
    if not good:
        _check_lora_add(y, x, a, b, scaling, adapters, cu, out, ws)
    if out is None:
        out = y
    if ws is None:
        nbytes = dgt_lora_workspace(tokens, requests, n, k, rank)
        ws = _made_on(stream, lambda: torch.empty(nbytes, dtype=torch.uint8, device=dev))
    _call("dgt_lora_add", dev, stream, y.data_ptr(), y_row, x.data_ptr(), x_row,
          a.data_ptr(), b.data_ptr(), scaling.data_ptr(), count, adapters.data_ptr(), cu.data_ptr(),
          requests, tokens, n, k, rank, out.data_ptr(), out.stride(0), ws.data_ptr(), ws.numel())
    return out
