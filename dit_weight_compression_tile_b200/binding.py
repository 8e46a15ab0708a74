"""Thin ctypes binding of libeptile.so (include/eptile.h): argument marshalling only.

Every step of compression runs in the library's C++ and every step of decompression in
its sm_100a kernel; this module passes torch tensors' pointers, sizes and streams.
There is no fallback: a missing library or a missing GPU raises ``EpError``.
"""
import contextlib
import ctypes as C
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libeptile.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "eptile.h")

BF16, FP16, FP32, INT8, FP8E4M3, LATTICE_I32 = 1, 2, 3, 4, 5, 6
TORCH_DTYPE = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32, INT8: torch.int8,
               FP8E4M3: torch.float8_e4m3fn}
CODE_OF = {v: k for k, v in TORCH_DTYPE.items()}
NAMES = {"bf16": BF16, "fp16": FP16, "fp32": FP32, "int8": INT8, "fp8_e4m3": FP8E4M3}


class EpError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        msg = lib().ep_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{what}: {msg} ({status})" if what else f"{msg} ({status})")


class Config(C.Structure):
    _fields_ = [("target_bpp", C.c_double), ("container_dtype", C.c_int32), ("blocks_per_lane", C.c_uint32),
                ("q_index", C.c_int32), ("n_threads", C.c_int32), ("coding", C.c_int32), ("layout", C.c_int32)]


class StreamInfo(C.Structure):
    _fields_ = [
        ("rows", C.c_int64), ("cols", C.c_int64),
        ("src_dtype", C.c_int32), ("container_dtype", C.c_int32),
        ("storage_nbytes", C.c_uint64), ("header_nbytes", C.c_uint64),
        ("actual_bpp", C.c_double), ("q_index", C.c_int32),
        ("n_tiles", C.c_uint32), ("blocks_per_lane", C.c_uint32),
        ("split", C.c_uint8 * 8), ("ntok", C.c_uint16 * 8),
        ("off_rowf", C.c_uint64), ("off_scales", C.c_uint64), ("off_freq", C.c_uint64),
        ("off_dir", C.c_uint64), ("off_tiles", C.c_uint64), ("out_nbytes", C.c_uint64),
        ("max_tile_nbytes", C.c_uint64), ("workspace_nbytes", C.c_uint64), ("paired", C.c_uint32),
        ("layout", C.c_uint32),
    ]

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def dtype(self):
        return TORCH_DTYPE[self.container_dtype]

    def storage_nbytes_(self, include_header=True):
        return self.storage_nbytes - (0 if include_header else self.header_nbytes)


class AnsConfig(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("blocks_per_lane", C.c_uint32), ("n_threads", C.c_int32),
                ("reserved", C.c_int32)]


class AnsInfo(C.Structure):
    _fields_ = [
        ("n_elems", C.c_int64), ("dtype", C.c_int32), ("ndim", C.c_int32), ("shape_", C.c_int64 * 8),
        ("storage_nbytes", C.c_uint64), ("ratio", C.c_double), ("n_tiles", C.c_uint32),
        ("blocks_per_lane", C.c_uint32), ("off_freq", C.c_uint64), ("off_dir", C.c_uint64),
        ("off_raw", C.c_uint64), ("off_tiles", C.c_uint64), ("out_nbytes", C.c_uint64),
        ("max_tile_nbytes", C.c_uint64), ("workspace_nbytes", C.c_uint64),
    ]

    @property
    def shape(self):
        return tuple(self.shape_[: self.ndim])

    @property
    def torch_dtype(self):
        return TORCH_DTYPE[self.dtype]


_lib = None


def declared_functions():
    """names of the functions include/eptile.h declares"""
    text = open(HEADER).read()
    return re.findall(r"^(?:int|size_t|const char \*)\s*\*?\s*(ep_\w+)\(", text, flags=re.M)


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m dit_weight_compression_tile_b200.build`")
        L = C.CDLL(LIB_PATH)
        p = C.c_void_p
        L.ep_compress_bound.restype = C.c_size_t
        L.ep_compress_bound.argtypes = [C.c_int64, C.c_int64, C.POINTER(Config)]
        L.ep_compress_device_scratch.restype = C.c_size_t
        L.ep_compress_device_scratch.argtypes = [C.c_int64, C.c_int64, C.POINTER(Config)]
        L.ep_compress_device.restype = C.c_int
        L.ep_compress_device.argtypes = [p, C.c_int32, C.c_int64, C.c_int64, C.POINTER(Config), p, C.c_size_t,
                                         C.POINTER(C.c_size_t), p, C.c_size_t, p]
        L.ep_compress_host.restype = C.c_int
        L.ep_compress_host.argtypes = [p, C.c_int32, C.c_int64, C.c_int64, C.POINTER(Config), p, C.c_size_t,
                                       C.POINTER(C.c_size_t)]
        L.ep_stream_info.restype = C.c_int
        L.ep_stream_info.argtypes = [p, C.c_size_t, C.POINTER(StreamInfo)]
        L.ep_prepare.restype = C.c_int
        L.ep_prepare.argtypes = [C.POINTER(StreamInfo), p, p, p, p]
        L.ep_decompress.restype = C.c_int
        L.ep_decompress.argtypes = [C.POINTER(StreamInfo), p, p, p, C.c_int32, p, p]
        L.ep_decompress_noalloc.restype = C.c_int
        L.ep_decompress_noalloc.argtypes = [C.POINTER(StreamInfo), p, p, C.c_int32, p, p]
        L.ep_decompress_host_scratch.restype = C.c_size_t
        L.ep_decompress_host_scratch.argtypes = [C.POINTER(StreamInfo), C.c_int32]
        L.ep_decompress_host.restype = C.c_int
        L.ep_decompress_host.argtypes = [C.POINTER(StreamInfo), p, p, C.c_int32, p, C.c_size_t, p, p]
        L.ep_linear_fused_workspace.restype = C.c_size_t
        L.ep_linear_fused_workspace.argtypes = [C.POINTER(StreamInfo), C.c_int64]
        L.ep_linear_fused_plan.restype = C.c_int
        L.ep_linear_fused_plan.argtypes = [C.POINTER(StreamInfo), C.c_int64, C.c_int32, C.POINTER(LinearPlan)]
        L.ep_linear_fused.restype = C.c_int
        L.ep_linear_fused.argtypes = [C.POINTER(StreamInfo), p, p, p, C.c_int64, p, p, p, C.c_size_t, p, p]
        L.ep_ans_compress_bound.restype = C.c_size_t
        L.ep_ans_compress_bound.argtypes = [C.c_int64, C.c_int32]
        L.ep_ans_compress_host.restype = C.c_int
        L.ep_ans_compress_host.argtypes = [p, C.c_int64, C.c_int32, p, C.POINTER(AnsConfig), p, C.c_size_t,
                                           C.POINTER(C.c_size_t)]
        L.ep_ans_stream_info.restype = C.c_int
        L.ep_ans_stream_info.argtypes = [p, C.c_size_t, C.POINTER(AnsInfo)]
        L.ep_ans_prepare.restype = C.c_int
        L.ep_ans_prepare.argtypes = [C.POINTER(AnsInfo), p, p, p, p]
        L.ep_ans_decompress.restype = C.c_int
        L.ep_ans_decompress.argtypes = [C.POINTER(AnsInfo), p, p, p, p, p]
        i32, i64 = C.c_int32, C.c_int64
        for name, args in (("ep_int4_quantize", [p, i32, i64, i64, i64, i32, p, p, i32, p]),
                           ("ep_int4_dequantize", [p, p, i32, i64, i64, i32, p, p]),
                           ("ep_int4_linear", [p, p, i64, i64, i32, i32, p, i64, i64, p, p, p, p]),
                           ("ep_int4_linear_dx", [p, p, i64, i64, i32, i32, p, i64, i64, p, p, p]),
                           ("ep_int4_scale_grad", [p, i64, p, p, i64, p, i64, i64, i32, i32, p, p, p]),
                           ("ep_act8_pack", [p, i32, i64, i64, i64, p, p, p]),
                           ("ep_act8_unpack", [p, p, i64, i64, p, i32, p])):
            getattr(L, name).restype = C.c_int
            getattr(L, name).argtypes = args
        L.ep_status_string.restype = C.c_char_p
        L.ep_status_string.argtypes = [C.c_int]
        _lib = L
    return _lib


CODING_AUTO, CODING_SINGLE, CODING_PAIRED = 0, 1, 2
LAYOUT_ROWS, LAYOUT_GEMM = 0, 1


def _config(target_bpp, container=0, blocks_per_lane=0, q_index=-1, n_threads=0, coding=CODING_AUTO,
            layout=LAYOUT_ROWS):
    if isinstance(container, str):
        container = NAMES[container]
    if isinstance(container, torch.dtype):
        container = CODE_OF[container]
    return Config(float(target_bpp), int(container or 0), int(blocks_per_lane), int(q_index), int(n_threads),
                  int(coding), int(layout))


def compress(tensor, target_bpp, container=0, blocks_per_lane=0, q_index=-1, n_threads=0, coding=CODING_AUTO,
             layout=LAYOUT_ROWS):
    """compress(tensor, config) on the host: returns the stream as a CPU uint8 tensor.

    ``tensor``: 2-D BF16/FP16/FP32 (moved to the CPU if needed).  ``container``: 0 (same as
    the source), a dtype code / name / torch dtype; INT8 and FP8 store per-row absmax codes.
    ``coding``: CODING_AUTO, CODING_SINGLE or CODING_PAIRED (ep_config.coding).  ``layout``:
    LAYOUT_ROWS, or LAYOUT_GEMM for tiles that are a consumer GEMM's 128 x 64 operand tiles."""
    if tensor.dim() != 2 or tensor.numel() == 0:
        raise EpError(-1, "compress needs a non-empty 2-D tensor")
    src = tensor.detach().to("cpu").contiguous()
    if src.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise EpError(-8, f"source dtype {src.dtype}")
    cfg = _config(target_bpp, container, blocks_per_lane, q_index, n_threads, coding, layout)
    L = lib()
    cap = L.ep_compress_bound(src.shape[0], src.shape[1], C.byref(cfg))
    out = torch.empty(max(cap, 64), dtype=torch.uint8)
    n = C.c_size_t(0)
    rc = L.ep_compress_host(src.data_ptr(), CODE_OF[src.dtype], src.shape[0], src.shape[1], C.byref(cfg),
                            out.data_ptr(), out.numel(), C.byref(n))
    if rc == -5:  # the bound is a guarantee; this is a second chance, not the normal path
        out = torch.empty(n.value, dtype=torch.uint8)
        rc = L.ep_compress_host(src.data_ptr(), CODE_OF[src.dtype], src.shape[0], src.shape[1], C.byref(cfg),
                                out.data_ptr(), out.numel(), C.byref(n))
    if rc != 0:
        raise EpError(rc, "ep_compress_host")
    return out[: n.value].clone()


def compress_device(tensor, target_bpp, container=0, blocks_per_lane=0, q_index=-1, stream=None,
                    coding=CODING_AUTO, layout=LAYOUT_ROWS):
    """compress(tensor, config) for a CUDA tensor (ep_compress_device): the same stream as
    ``compress`` byte for byte, built on the GPU.  Returns a CUDA uint8 tensor."""
    if tensor.dim() != 2 or tensor.numel() == 0:
        raise EpError(-1, "compress needs a non-empty 2-D tensor")
    if not tensor.is_cuda:
        raise EpError(-1, "compress_device needs a CUDA tensor")
    src = tensor.detach().contiguous()
    if src.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise EpError(-8, f"source dtype {src.dtype}")
    cfg = _config(target_bpp, container, blocks_per_lane, q_index, 0, coding, layout)
    L = lib()
    R, Cc = src.shape
    scratch = torch.empty(max(1, L.ep_compress_device_scratch(R, Cc, C.byref(cfg))), dtype=torch.uint8,
                          device=src.device)
    cap = L.ep_compress_bound(R, Cc, C.byref(cfg))
    out = torch.empty(max(cap, 64), dtype=torch.uint8, device=src.device)
    n = C.c_size_t(0)
    s = (stream or torch.cuda.current_stream(src.device)).cuda_stream
    rc = L.ep_compress_device(src.data_ptr(), CODE_OF[src.dtype], R, Cc, C.byref(cfg), out.data_ptr(), out.numel(),
                              C.byref(n), scratch.data_ptr(), scratch.numel(), s)
    if rc != 0:
        raise EpError(rc, "ep_compress_device")
    return out[: n.value].clone()


def stream_info(blob):
    """CompressedTensor properties from a host copy of the stream (CPU uint8 tensor)."""
    b = blob.detach().to("cpu").contiguous()
    info = StreamInfo()
    rc = lib().ep_stream_info(b.data_ptr(), b.numel(), C.byref(info))
    if rc != 0:
        raise EpError(rc, "ep_stream_info")
    return info


def prepare(d_blob, info=None, workspace=None, status=None, stream=None):
    """The decoder's slot tables for one device copy of a stream (ep_prepare): run once when the
    stream lands on the device.  Returns the workspace (CUDA uint8 tensor of
    ``info.workspace_nbytes``), allocated here unless ``workspace`` is given."""
    if not d_blob.is_cuda:
        raise EpError(-1, "prepare needs the stream in device memory")
    if info is None:
        info = stream_info(d_blob.cpu())
    if workspace is None:
        workspace = torch.empty(info.workspace_nbytes, dtype=torch.uint8, device=d_blob.device)
    if (not workspace.is_cuda or workspace.dtype != torch.uint8 or workspace.numel() < info.workspace_nbytes
            or not workspace.is_contiguous()):
        raise EpError(-1, "workspace does not match the stream")
    st = status.data_ptr() if status is not None else None
    s = (stream or torch.cuda.current_stream(d_blob.device)).cuda_stream
    rc = lib().ep_prepare(C.byref(info), d_blob.data_ptr(), workspace.data_ptr(), st, s)
    if rc != 0:
        raise EpError(rc, "ep_prepare")
    return workspace


def dtype_code(d):
    """EP_* dtype code of a torch dtype, a name ("bf16", ...) or a code"""
    if isinstance(d, torch.dtype):
        if d not in CODE_OF:
            raise EpError(-1, f"no container dtype for {d}")
        return CODE_OF[d]
    if isinstance(d, str):
        return NAMES[d]
    return int(d)


def decompress(d_blob, info=None, workspace=None, out=None, status=None, stream=None, lattice=False,
               out_dtype=None):
    """decompress(compressed): the fused GPU decode of a device-resident stream.

    ``d_blob``: CUDA uint8 tensor holding the whole stream.  ``info``: from ``stream_info``
    (parsed from ``d_blob`` through a host copy when omitted).  ``workspace``: from ``prepare``
    on this ``d_blob``.  When omitted, every call allocates a workspace and runs ``prepare``
    again on the same stream (a few microseconds of table building per call); callers that
    decode one stream repeatedly should prepare once and pass the workspace, as
    ``CompressedTensor`` does.  ``out``: optional CUDA
    tensor of ``info.shape`` / ``info.dtype``.  ``status``: optional CUDA int32 tensor of one
    element into which damage flags are ORed.  Launches on ``stream`` (default: the current
    stream).  ``lattice=True`` returns the decoded lattice points v = 2z (int32) instead of
    weights.  ``out_dtype``: for a BF16 / FP16 / FP32 container, any of the three (the fp32
    weight rounded once into it); default the container's dtype."""
    if not d_blob.is_cuda:
        raise EpError(-1, "decompress needs the stream in device memory")
    if info is None:
        info = stream_info(d_blob.cpu())
    if workspace is None:
        workspace = prepare(d_blob, info, status=status, stream=stream)
    dt = LATTICE_I32 if lattice else (info.container_dtype if out_dtype is None else dtype_code(out_dtype))
    want = torch.int32 if lattice else TORCH_DTYPE.get(dt)
    if want is None:
        raise EpError(-1, f"output dtype code {dt}")
    if out is None:
        out = torch.empty(info.shape, dtype=want, device=d_blob.device)
    if not out.is_cuda or out.dtype != want or tuple(out.shape) != info.shape or not out.is_contiguous():
        raise EpError(-1, "output tensor does not match the stream")
    st = status.data_ptr() if status is not None else None
    s = (stream or torch.cuda.current_stream(d_blob.device)).cuda_stream
    rc = lib().ep_decompress(C.byref(info), d_blob.data_ptr(), workspace.data_ptr(), out.data_ptr(), dt, st, s)
    if rc != 0:
        raise EpError(rc, "ep_decompress")
    return out


def decompress_host_scratch(info, out_dtype=None):
    """bytes of device scratch that ``decompress_host`` needs (ep_decompress_host_scratch)"""
    dt = info.container_dtype if out_dtype is None else dtype_code(out_dtype)
    return int(lib().ep_decompress_host_scratch(C.byref(info), dt))


def decompress_host(h_blob, info=None, out=None, out_dtype=None, scratch=None, status=None, stream=None,
                    device=None, sync=True):
    """decompress(compressed) for a stream in host memory (ep_decompress_host): the stream is
    copied to the GPU, decoded by the fused kernel there and the weights copied back into a host
    tensor, all on one CUDA stream.  ``h_blob``: CPU uint8 tensor (pinned memory lets the copies
    run without staging).  ``out``: optional CPU tensor of ``info.shape`` and the output dtype.
    ``scratch``: optional CUDA uint8 tensor of ``decompress_host_scratch`` bytes, allocated on
    ``device`` (default: the current CUDA device) when omitted.  With ``sync`` the call waits for
    the stream before returning; otherwise ``out`` is valid once ``stream`` has been synchronised."""
    if h_blob.is_cuda or h_blob.dtype != torch.uint8 or not h_blob.is_contiguous():
        raise EpError(-1, "decompress_host takes the stream as a contiguous CPU uint8 tensor")
    if not torch.cuda.is_available():
        raise EpError(-1, "decompress_host decodes on a CUDA device and none is available")
    if info is None:
        info = stream_info(h_blob)
    dt = info.container_dtype if out_dtype is None else dtype_code(out_dtype)
    want = TORCH_DTYPE.get(dt)
    if want is None:
        raise EpError(-1, f"output dtype code {dt}")
    if out is None:
        out = torch.empty(info.shape, dtype=want, pin_memory=True)
    if out.is_cuda or out.dtype != want or tuple(out.shape) != info.shape or not out.is_contiguous():
        raise EpError(-1, "output tensor does not match the stream")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    need = decompress_host_scratch(info, dt)
    if scratch is None:
        scratch = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if not scratch.is_cuda or scratch.dtype != torch.uint8 or scratch.numel() < need:
        raise EpError(-1, "scratch does not match the stream")
    st = status.data_ptr() if status is not None else None
    cs = stream or torch.cuda.current_stream(scratch.device)
    with torch.cuda.device(scratch.device):
        rc = lib().ep_decompress_host(C.byref(info), h_blob.data_ptr(), out.data_ptr(), dt, scratch.data_ptr(),
                                      scratch.numel(), st, cs.cuda_stream)
    if rc != 0:
        raise EpError(rc, "ep_decompress_host")
    if sync:
        cs.synchronize()
    return out


# ---------------------------------------------------------------- the Tile-ANS lossless scheme
def ans_compress(tensor, blocks_per_lane=0, n_threads=0):
    """compress(tensor, TileANSConfig()) on the host (ep_ans_compress_host): every bit of a BF16,
    FP16, FP32, INT8 or FP8 E4M3 tensor of any shape (1 to 8 dims).  Returns the stream as a CPU
    uint8 tensor."""
    if tensor.dtype not in CODE_OF:
        raise EpError(-1, f"Tile-ANS takes BF16, FP16, FP32, INT8 or FP8 E4M3, not {tensor.dtype}")
    if tensor.numel() == 0 or tensor.dim() < 1 or tensor.dim() > 8:
        raise EpError(-1, "Tile-ANS needs a non-empty tensor of 1 to 8 dims")
    src = tensor.detach().to("cpu").contiguous()
    cfg = AnsConfig(CODE_OF[src.dtype], int(blocks_per_lane), int(n_threads), 0)
    dims = (C.c_int64 * 8)(*src.shape)
    L = lib()
    cap = L.ep_ans_compress_bound(src.numel(), cfg.dtype)
    out = torch.empty(max(cap, 1024), dtype=torch.uint8)
    n = C.c_size_t(0)
    rc = L.ep_ans_compress_host(src.data_ptr(), src.numel(), src.dim(), dims, C.byref(cfg), out.data_ptr(),
                                out.numel(), C.byref(n))
    if rc == -5:
        out = torch.empty(n.value, dtype=torch.uint8)
        rc = L.ep_ans_compress_host(src.data_ptr(), src.numel(), src.dim(), dims, C.byref(cfg), out.data_ptr(),
                                    out.numel(), C.byref(n))
    if rc != 0:
        raise EpError(rc, "ep_ans_compress_host")
    return out[: n.value].clone()


def ans_stream_info(blob):
    b = blob.detach().to("cpu").contiguous()
    info = AnsInfo()
    rc = lib().ep_ans_stream_info(b.data_ptr(), b.numel(), C.byref(info))
    if rc != 0:
        raise EpError(rc, "ep_ans_stream_info")
    return info


def ans_prepare(d_blob, info, workspace=None, status=None, stream=None):
    """the decoder's slot table for one device copy of a Tile-ANS stream (ep_ans_prepare)"""
    if not d_blob.is_cuda:
        raise EpError(-1, "ans_prepare needs the stream in device memory")
    if workspace is None:
        workspace = torch.empty(info.workspace_nbytes, dtype=torch.uint8, device=d_blob.device)
    if not workspace.is_cuda or workspace.numel() < info.workspace_nbytes:
        raise EpError(-1, "workspace does not match the stream")
    st = status.data_ptr() if status is not None else None
    s = (stream or torch.cuda.current_stream(d_blob.device)).cuda_stream
    rc = lib().ep_ans_prepare(C.byref(info), d_blob.data_ptr(), workspace.data_ptr(), st, s)
    if rc != 0:
        raise EpError(rc, "ep_ans_prepare")
    return workspace


def ans_decompress(d_blob, info, workspace=None, out=None, status=None, stream=None):
    """decompress of a device-resident Tile-ANS stream (ep_ans_decompress): the tensor, bit for bit.
    Without ``workspace`` the table is prepared here on every call."""
    if not d_blob.is_cuda:
        raise EpError(-1, "ans_decompress needs the stream in device memory")
    if workspace is None:
        workspace = ans_prepare(d_blob, info, status=status, stream=stream)
    want = TORCH_DTYPE[info.dtype]
    if out is None:
        out = torch.empty(info.shape, dtype=want, device=d_blob.device)
    if not out.is_cuda or out.dtype != want or tuple(out.shape) != info.shape or not out.is_contiguous():
        raise EpError(-1, "output tensor does not match the stream")
    st = status.data_ptr() if status is not None else None
    s = (stream or torch.cuda.current_stream(d_blob.device)).cuda_stream
    rc = lib().ep_ans_decompress(C.byref(info), d_blob.data_ptr(), workspace.data_ptr(), out.data_ptr(), st, s)
    if rc != 0:
        raise EpError(rc, "ep_ans_decompress")
    return out


# ---------------------------------------------------------------- the decode fused into a GEMM
class LinearPlan(C.Structure):
    """ep_linear_plan: the launch ep_linear_fused would make (grid, warps, shared-memory layout)"""
    _fields_ = [(n, C.c_uint32) for n in ("bands", "ctas", "tiles_per_cta", "accumulators", "spread", "splits",
                                          "decoding_warps", "threads",
                                          "tokens_padded", "tmem_columns", "tile_buffer_bytes", "smem_tables_bytes",
                                          "smem_barriers_offset", "smem_tiles_offset", "smem_slices_offset",
                                          "smem_x_offset", "smem_x_bytes_per_warp")] + \
               [("smem_bytes", C.c_uint64), ("work_bytes", C.c_uint64)]


def linear_fused_plan(info, m, sms):
    """(status, LinearPlan) of ep_linear_fused for m tokens on a GPU with `sms` multiprocessors,
    computed on the host"""
    plan = LinearPlan()
    rc = lib().ep_linear_fused_plan(C.byref(info), m, sms, C.byref(plan))
    return rc, plan


def linear_fused_workspace(info, m):
    """bytes of scratch ep_linear_fused needs for m tokens (0: the stream or m is not one it takes)"""
    return int(lib().ep_linear_fused_workspace(C.byref(info), m))


def linear_fused(x, d_blob, info, tables, bias=None, out=None, work=None, status=None, stream=None):
    """Y = X W^T (+ bias) with W decoded inside the tcgen05 GEMM (ep_linear_fused).  ``x``: CUDA
    BF16 (m, K) with 1 <= m <= 128; ``d_blob``: a GEMM-ordered (LAYOUT_GEMM) BF16, INT8 or FP8
    stream on the device (INT8 / FP8: the activations are quantized per token and the codes
    multiplied); ``tables``: from ``prepare``; ``work``: scratch of linear_fused_workspace bytes,
    zero-filled before its first use (the call leaves it reusable; a new one is zero-allocated
    when absent or too small).  Returns the BF16 (m, N) output."""
    if not (x.is_cuda and d_blob.is_cuda and tables.is_cuda):
        raise EpError(-1, "linear_fused works on CUDA tensors")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != info.cols:
        raise EpError(-1, "x must be a BF16 (m, in_features) tensor")
    x = x.contiguous()
    m = x.shape[0]
    L = lib()
    need = linear_fused_workspace(info, m)
    if need == 0:
        raise EpError(-1, "ep_linear_fused takes a GEMM-ordered BF16 / INT8 / FP8 stream and 1 <= m <= 128")
    if work is None or work.numel() * work.element_size() < need:
        work = torch.zeros(need, dtype=torch.uint8, device=x.device)
    elif not (work.is_cuda and work.is_contiguous()):
        raise EpError(-1, "work must be a contiguous CUDA tensor")
    if out is None:
        out = torch.empty((m, info.rows), dtype=torch.bfloat16, device=x.device)
    elif not (out.is_cuda and out.dtype == torch.bfloat16 and out.is_contiguous() and out.numel() == m * info.rows):
        raise EpError(-1, "out must be a contiguous CUDA BF16 tensor of m x out_features elements")
    if bias is not None:
        bias = bias.contiguous()
        if not bias.is_cuda or bias.dtype != torch.bfloat16 or bias.numel() != info.rows:
            raise EpError(-1, "bias must be a CUDA BF16 tensor with out_features elements")
    st = status.data_ptr() if status is not None else None
    s = (stream or torch.cuda.current_stream(x.device)).cuda_stream
    rc = L.ep_linear_fused(C.byref(info), d_blob.data_ptr(), tables.data_ptr(), x.data_ptr(), m,
                           bias.data_ptr() if bias is not None else None, out.data_ptr(), work.data_ptr(),
                           work.numel() * work.element_size(), st, s)
    if rc != 0:
        raise EpError(rc, "ep_linear_fused")
    return out


# ---------------------------------------------------------------- 4-bit weights with group scales
INT4_GROUPS = (32, 64, 128)
ACT8_GROUP = 128  # features per scale of an activation checkpoint
INT4_STREAM_TOKENS = 16  # ep_int4_linear streams the weight for up to so many tokens (any rows will do)
_INT4_DTYPES = (torch.bfloat16, torch.float16)


# the current stream's handle without building a Stream object around it, and the current device without
# a look at whether CUDA is up (with CUDA tensors in hand it is): 1.5 us of a call of 10
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_tracing = getattr(torch._C, "_is_tracing", None) or torch.jit.is_tracing


def _refuse_trace(name):
    """a trace would record the allocation of the output and not the kernel that fills it"""
    raise EpError(-1, f"{name} cannot be traced: int4_group_linear and GroupedINT4Linear can")


def _elsewhere(t, stream):
    """whether a call on ``t`` must first make a device or a stream current"""
    return stream is not None or _current_device() != t.device.index


@contextlib.contextmanager
def _made_current(t, stream):
    """``t``'s device and ``stream`` (if given) as the current ones: what a call allocates belongs to the
    stream that it launches on"""
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield


def _rows(t):
    """``t`` (2-D) with contiguous rows, and the distance between them"""
    m, k = t.shape
    ld, one = t.stride()
    if (k > 1 and one != 1) or (m > 1 and ld < k):
        t = t.detach().contiguous()
        ld = k
    return t, (ld if m > 1 else k)


def _aligned_rows(t, ld):
    """``t`` and its rows' distance, copied into rows that begin on 16 bytes if they do not"""
    if ld % 8 or t.data_ptr() % 16:
        m, k = t.shape
        ld = (k + 7) // 8 * 8
        t = t.new_empty((m, ld))[:, :k].copy_(t.detach())
    return t, ld


def _tiles(t):
    """``_rows`` for the tensor-core products: those copy rows that begin on 16 bytes by TMA, others element
    by element, so a large ``t`` that does not lie that way is first copied into rows that do (2048 x 8191
    BF16: 3.3 ms against 0.2 ms; below 2^17 elements the copy costs more than it saves)"""
    t, ld = _rows(t)
    return _aligned_rows(t, ld) if t.numel() >= 1 << 17 else (t, ld)


def _stream_rows(t, weights):
    """``_rows`` for the product that streams the weight: the same where the weight is large (5 tokens: 8192 x
    28671 33.8 us, 72.5 without the copy, at 2^26 weights 16.0 against 24.4; the copy costs the host 5 us, and smaller
    products are bound by the host's 10; in a CUDA graph, where they are not, rows on 16 bytes are the caller's to lay
    out)"""
    t, ld = _rows(t)
    return _aligned_rows(t, ld) if t.shape[0] > 1 and weights >= 1 << 26 else (t, ld)


def _int4_weight(codes, scales, in_features, group):
    """checks a weight's codes and scales against each other; returns out_features"""
    if group not in INT4_GROUPS:
        raise EpError(-1, f"group must be one of {INT4_GROUPS}, not {group}")
    if in_features < 1:
        raise EpError(-1, "in_features must be at least 1")
    row = (in_features + 31) // 32 * 16
    if not codes.is_cuda or codes.dtype != torch.uint8 or codes.dim() != 2 or codes.shape[1] != row or codes.shape[0] < 1 \
            or not codes.is_contiguous():
        raise EpError(-1, f"codes must be a contiguous CUDA uint8 tensor of {row} bytes per row")
    n = codes.shape[0]
    if scales is not None and (scales.dtype not in _INT4_DTYPES or scales.shape != (n, -(-in_features // group))
                               or not scales.is_contiguous() or scales.device != codes.device):
        raise EpError(-1, f"scales must be contiguous BF16 or FP16 of shape {(n, -(-in_features // group))} on the codes' "
                          "device")
    return n


def _output(out, like, shape, dtype):
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if out.device != like.device or out.dtype != dtype or out.shape != shape or not out.is_contiguous():
        raise EpError(-1, f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on {like.device}")
    return out


def _status(status, like):
    if status is None:
        return None
    if status.device != like.device or status.dtype != torch.int32 or status.numel() < 1:
        raise EpError(-1, "status must be an int32 tensor on the call's device")
    return status.data_ptr()


def int4_quantize(weight, group=128, dtype=None, stream=None):
    """(codes, scales) of a CUDA BF16 / FP16 / FP32 (out_features, in_features) weight (ep_int4_quantize):
    codes uint8 (out_features, ceil(in_features / 32) * 16), scales (out_features, ceil(in_features /
    group)) of ``dtype`` (torch.bfloat16 or torch.float16; default the weight's, BF16 for FP32)."""
    if _tracing():
        _refuse_trace("int4_quantize")
    if weight.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise EpError(-8, f"source dtype {weight.dtype}")
    if not weight.is_cuda or weight.dim() != 2 or weight.numel() == 0:
        raise EpError(-1, "weight must be a non-empty 2-D CUDA tensor")
    if group not in INT4_GROUPS:
        raise EpError(-1, f"group must be one of {INT4_GROUPS}, not {group}")
    if dtype is None:
        dtype = torch.bfloat16 if weight.dtype == torch.float32 else weight.dtype
    if dtype not in _INT4_DTYPES:
        raise EpError(-1, f"scales are BF16 or FP16, not {dtype}")
    if _elsewhere(weight, stream):
        with _made_current(weight, stream):
            return int4_quantize(weight, group, dtype)
    w, ld = _rows(weight)
    n, k = w.shape
    codes = w.new_empty((n, (k + 31) // 32 * 16), dtype=torch.uint8)
    scales = w.new_empty((n, -(-k // group)), dtype=dtype)
    rc = lib().ep_int4_quantize(w.data_ptr(), CODE_OF[w.dtype], n, k, ld, group, codes.data_ptr(), scales.data_ptr(),
                                CODE_OF[dtype], _raw_stream(w.device.index))
    if rc != 0:
        raise EpError(rc, "ep_int4_quantize")
    return codes, scales


def int4_dequantize(codes, scales, in_features, group=128, out=None, stream=None):
    """the (out_features, in_features) weight s q in the scales' dtype (ep_int4_dequantize)"""
    if _tracing():
        _refuse_trace("int4_dequantize")
    if scales is None:
        raise EpError(-1, "scales are needed")
    n = _int4_weight(codes, scales, in_features, group)
    if _elsewhere(codes, stream):
        with _made_current(codes, stream):
            return int4_dequantize(codes, scales, in_features, group, out)
    out = _output(out, codes, (n, in_features), scales.dtype)
    rc = lib().ep_int4_dequantize(codes.data_ptr(), scales.data_ptr(), CODE_OF[scales.dtype], n, in_features, group,
                                  out.data_ptr(), _raw_stream(codes.device.index))
    if rc != 0:
        raise EpError(rc, "ep_int4_dequantize")
    return out


def _int4_linear_check(x, codes, scales, group, bias):
    """checks the arguments of a forward; returns out_features"""
    if x.dim() != 2 or scales is None:
        raise EpError(-1, "x must be a 2-D CUDA tensor, and scales are needed")
    k = x.shape[1]
    dtype, device = x.dtype, x.device
    if codes.dim() == 2 and k > 0 and group in INT4_GROUPS and dtype in _INT4_DTYPES and device.type == "cuda":
        n = codes.shape[0]
        if (n > 0 and codes.shape[1] == (k + 31) // 32 * 16 and codes.dtype == torch.uint8 and codes.device == device
                and codes.is_contiguous() and scales.shape == (n, -(-k // group)) and scales.dtype == dtype
                and scales.device == device and scales.is_contiguous()
                and (bias is None or (bias.shape == (n,) and bias.dtype == dtype and bias.device == device
                                      and bias.is_contiguous()))):
            return n
    # something is wrong: say what
    n = _int4_weight(codes, scales, k, group)
    if dtype != scales.dtype or device != codes.device:
        raise EpError(-1, f"x must be {scales.dtype} on {codes.device}, as the scales are")
    raise EpError(-1, f"bias must be {n} contiguous {dtype} elements on {device}")


# The calls themselves, on checked arguments with the device and stream current
def _launch_linear(x, codes, scales, n, group, bias, out, status):
    m, k = x.shape
    x, ld = _tiles(x) if m > INT4_STREAM_TOKENS else _stream_rows(x, n * k)
    rc = lib().ep_int4_linear(codes.data_ptr(), scales.data_ptr(), n, k, group, CODE_OF[x.dtype], x.data_ptr(), m, ld,
                              None if bias is None else bias.data_ptr(), out.data_ptr(), status,
                              _raw_stream(x.device.index))
    if rc != 0:
        raise EpError(rc, "ep_int4_linear")
    return out


def _launch_dx(dy, ld, codes, scales, k, group, out, status):
    m, n = dy.shape
    rc = lib().ep_int4_linear_dx(codes.data_ptr(), scales.data_ptr(), n, k, group, CODE_OF[dy.dtype], dy.data_ptr(), m, ld,
                                 out.data_ptr(), status, _raw_stream(dy.device.index))
    if rc != 0:
        raise EpError(rc, "ep_int4_linear_dx")
    return out


def _launch_pack(x):
    m, k = x.shape
    codes = x.new_empty((m, (k + 15) // 16 * 16), dtype=torch.int8)
    scales = x.new_empty((m, -(-k // ACT8_GROUP)), dtype=torch.float32)
    x, ld = _rows(x)
    rc = lib().ep_act8_pack(x.data_ptr(), CODE_OF[x.dtype], m, k, ld, codes.data_ptr(), scales.data_ptr(),
                            _raw_stream(x.device.index))
    if rc != 0:
        raise EpError(rc, "ep_act8_pack")
    return codes, scales


def _launch_scale_grad(dy, ld, act_codes, act_scales, codes, k, group, out, status):  # (the checkpoint: addresses)
    m, n = dy.shape
    rc = lib().ep_int4_scale_grad(dy.data_ptr(), ld, act_codes, act_scales, m, codes.data_ptr(), n, k, group,
                                  CODE_OF[dy.dtype], out.data_ptr(), status, _raw_stream(dy.device.index))
    if rc != 0:
        raise EpError(rc, "ep_int4_scale_grad")
    return out


def int4_layer_forward(x, codes, scales, group, bias, checkpoint, status=None):
    """``int4_linear`` and, with ``checkpoint``, ``act8_pack`` of its input, checked once: (y, act), act one
    int8 tensor with the checkpoint's codes and, from the next multiple of 16 bytes, its scales, or None"""
    n = _int4_linear_check(x, codes, scales, group, bias)
    if _elsewhere(x, None):
        with _made_current(x, None):
            return int4_layer_forward(x, codes, scales, group, bias, checkpoint, status)
    m, k = x.shape
    y = _launch_linear(x, codes, scales, n, group, bias, x.new_empty((m, n)), _status(status, x))
    if not checkpoint:
        return y, None
    size = int(m * ((k + 15) // 16 * 16))  # (a trace's sizes are tensors, and no offsets of an address)
    act = x.new_empty(size + 4 * m * -(-k // ACT8_GROUP), dtype=torch.int8)
    x, ld = _rows(x)
    at = act.data_ptr()
    rc = lib().ep_act8_pack(x.data_ptr(), CODE_OF[x.dtype], m, k, ld, at, at + size, _raw_stream(x.device.index))
    if rc != 0:
        raise EpError(rc, "ep_act8_pack")
    return y, act


def int4_layer_backward(dy, act, codes, scales, in_features, group, input_grad, scale_grad, status=None):
    """the gradients (dx, ds) that are asked for (None otherwise) of ``int4_layer_forward``'s y, from what it
    was given and gave: these are not checked again"""
    if _elsewhere(dy, None):
        with _made_current(dy, None):
            return int4_layer_backward(dy, act, codes, scales, in_features, group, input_grad, scale_grad, status)
    dy, ld = _tiles(dy)
    dx = ds = None
    status = None if status is None else status.data_ptr()
    if input_grad:
        dx = _launch_dx(dy, ld, codes, scales, in_features, group, dy.new_empty((dy.shape[0], in_features)), status)
    if scale_grad:
        at = act.data_ptr()
        ds = _launch_scale_grad(dy, ld, at, at + dy.shape[0] * ((in_features + 15) // 16 * 16), codes, in_features, group,
                                dy.new_empty(scales.shape), status)
    return dx, ds


def int4_linear(x, codes, scales, group=128, bias=None, out=None, status=None, stream=None):
    """Y = X W^T (+ bias) with a 4-bit group-scaled W (ep_int4_linear).  ``x``: CUDA (m, in_features) of the
    scales' dtype, any m, rows any distance apart; ``codes``, ``scales``: from ``int4_quantize``.  Returns
    the contiguous (m, out_features) output."""
    if _tracing():
        _refuse_trace("int4_linear")
    n = _int4_linear_check(x, codes, scales, group, bias)
    if _elsewhere(x, stream):
        with _made_current(x, stream):
            return int4_linear(x, codes, scales, group, bias, out, status)
    return _launch_linear(x, codes, scales, n, group, bias, _output(out, x, (x.shape[0], n), x.dtype), _status(status, x))


def int4_linear_dx(dy, codes, scales, in_features, group=128, out=None, status=None, stream=None):
    """dX = dY W, the input gradient of ``int4_linear`` (ep_int4_linear_dx).  ``dy``: CUDA (m,
    out_features) of the scales' dtype."""
    if _tracing():
        _refuse_trace("int4_linear_dx")
    if scales is None:
        raise EpError(-1, "scales are needed")
    n = _int4_weight(codes, scales, in_features, group)
    if dy.dim() != 2 or dy.shape[1] != n or dy.dtype != scales.dtype or dy.device != codes.device:
        raise EpError(-1, f"dy must be (m, {n}) of {scales.dtype} on {codes.device}, as the scales are")
    if _elsewhere(dy, stream):
        with _made_current(dy, stream):
            return int4_linear_dx(dy, codes, scales, in_features, group, out, status)
    dy, ld = _tiles(dy)
    return _launch_dx(dy, ld, codes, scales, in_features, group, _output(out, dy, (dy.shape[0], in_features), dy.dtype),
                      _status(status, dy))


def act8_pack(x, stream=None):
    """(codes, scales) of an 8-bit checkpoint of CUDA BF16 / FP16 / FP32 (m, features) activations
    (ep_act8_pack): codes int8 (m, ceil(features / 16) * 16), scales fp32 (m, ceil(features / 128))."""
    if _tracing():
        _refuse_trace("act8_pack")
    if x.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise EpError(-8, f"source dtype {x.dtype}")
    if not x.is_cuda or x.dim() != 2 or x.shape[1] < 1:
        raise EpError(-1, "x must be a 2-D CUDA tensor with at least one feature")
    if _elsewhere(x, stream):
        with _made_current(x, stream):
            return act8_pack(x)
    return _launch_pack(x)


def _act8(codes, scales, features):
    row = (features + 15) // 16 * 16
    if features < 1 or not codes.is_cuda or codes.dtype != torch.int8 or codes.dim() != 2 or codes.shape[1] != row \
            or not codes.is_contiguous():
        raise EpError(-1, f"checkpoint codes must be contiguous CUDA int8 rows of {row} bytes")
    if scales.dtype != torch.float32 or scales.shape != (codes.shape[0], -(-features // ACT8_GROUP)) \
            or not scales.is_contiguous() or scales.device != codes.device:
        raise EpError(-1, "checkpoint scales must be contiguous fp32 of shape "
                          f"{(codes.shape[0], -(-features // ACT8_GROUP))}")


def act8_unpack(codes, scales, features, dtype=torch.bfloat16, out=None, stream=None):
    """the (m, features) activations a c of a checkpoint, rounded once to ``dtype`` (ep_act8_unpack)"""
    if _tracing():
        _refuse_trace("act8_unpack")
    _act8(codes, scales, features)
    if dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise EpError(-8, f"output dtype {dtype}")
    if _elsewhere(codes, stream):
        with _made_current(codes, stream):
            return act8_unpack(codes, scales, features, dtype, out)
    m = codes.shape[0]
    out = _output(out, codes, (m, features), dtype)
    rc = lib().ep_act8_unpack(codes.data_ptr(), scales.data_ptr(), m, features, out.data_ptr(), CODE_OF[dtype],
                              _raw_stream(codes.device.index))
    if rc != 0:
        raise EpError(rc, "ep_act8_unpack")
    return out


def int4_scale_grad(dy, act_codes, act_scales, codes, in_features, group=128, out=None, status=None, stream=None):
    """the gradient of every group scale of ``int4_linear`` (ep_int4_scale_grad): ``dy`` CUDA BF16 / FP16
    (m, out_features), the forward's input as an 8-bit checkpoint (``act8_pack``), the weight's codes.
    Returns (out_features, ceil(in_features / group)) in dy's dtype."""
    if _tracing():
        _refuse_trace("int4_scale_grad")
    n = _int4_weight(codes, None, in_features, group)
    _act8(act_codes, act_scales, in_features)
    if dy.dtype not in _INT4_DTYPES or dy.dim() != 2 or dy.shape[1] != n:
        raise EpError(-1, f"dy must be (m, {n}) of BF16 or FP16")
    if dy.device != codes.device or act_codes.device != codes.device or dy.shape[0] != act_codes.shape[0]:
        raise EpError(-1, "dy, the checkpoint and the codes must be of the same tokens on one device")
    if _elsewhere(dy, stream):
        with _made_current(dy, stream):
            return int4_scale_grad(dy, act_codes, act_scales, codes, in_features, group, out, status)
    dy, ld = _tiles(dy)
    return _launch_scale_grad(dy, ld, act_codes.data_ptr(), act_scales.data_ptr(), codes, in_features, group,
                              _output(out, dy, (n, -(-in_features // group)), dy.dtype), _status(status, dy))
