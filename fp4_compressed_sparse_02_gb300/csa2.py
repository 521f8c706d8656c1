"""Python face of the CSA2 C ABI: torch tensors in, device pointers to libcsa2.so.

Names follow include/csa2.h: compress_quant, index_full, index_reindex, sparse_attn, and the
operators around them: rms_norm, rope, rope_table, fp4_quant, fp4_linear, and, for the model's plain
attention layers, page_plan, kv8_append, kv8_select, kv8_attn.
PyTorch provides device memory and the current stream; every computation runs in the
library's kernels.  Outputs are allocated here when the caller passes none (pass them
in, together with a pre-sized Workspace, to capture calls in a CUDA graph).
"""
import ctypes
import math
import struct
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib

PAGE = 64
BF16, F32, FP8E4M3, FP4E2M1X2 = 0, 1, 2, 3


def _on_device(t, dev, name):
    """Refuse a tensor that is not on CUDA device number dev."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if at != dev:
        raise ValueError(f"{name}: on cuda:{at}, but the call's tensors are on cuda:{dev}")


def _pointers(device):
    """ptr(t): the address of a contiguous tensor on this device, None of None."""
    dev = device.index

    def ptr(t: Optional[torch.Tensor]):
        if t is None:
            return None
        if t.get_device() != dev:
            _on_device(t, dev, "operand")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        return ctypes.c_void_p(t.data_ptr())

    return ptr


def _expect(t, dtypes, name):
    if t is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")


_I32 = (torch.int32,)
_B16 = (torch.bfloat16, torch.int16)
_U8 = (torch.uint8,)
_F32 = (torch.float32,)


def _stream(dev):
    """Handle of CUDA device number dev's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev)


_gpus = 0                                  # how many the process has (asked at the first call)


def _is_current(dev):
    """Whether CUDA device number dev is the current one: a launch goes to that, whatever device its stream's handle and
    its pointers belong to."""
    global _gpus
    if not _gpus:
        _gpus = torch.cuda.device_count()
    return _gpus == 1 or dev == torch._C._cuda_getDevice()


@dataclass
class PagedCache:
    """Paged Main KV planes: codes uint8 [pages, 64, d/2], scales uint8 [pages, 64, d/16],
    page_table int32 [seqs, max_pages], and indexer K in one of two forms: idx_k bf16
    [pages, 64, d_ik], or (compressed) idx_k8 uint8 E4M3 [pages, 64, d_ik] with
    idx_k8_scale float32 [pages, 64].  The FP8 form is used when idx_k8 is set."""
    codes: torch.Tensor
    scales: torch.Tensor
    idx_k: Optional[torch.Tensor]
    page_table: torch.Tensor
    idx_k8: Optional[torch.Tensor] = None
    idx_k8_scale: Optional[torch.Tensor] = None

    @property
    def d(self):
        return self.codes.shape[-1] * 2

    @property
    def d_ik(self):
        if self.idx_k8 is not None:
            return self.idx_k8.shape[-1]
        return self.idx_k.shape[-1] if self.idx_k is not None else 0

    @property
    def num_pages(self):
        return self.codes.shape[0]

    @property
    def num_seqs(self):
        return self.page_table.shape[0]

    @property
    def max_pages(self):
        return self.page_table.shape[1]

    @staticmethod
    def allocate(num_seqs, entries_per_seq, d, d_ik, device, page_table=None, idx_k_fp8=False):
        mp = (entries_per_seq + PAGE - 1) // PAGE
        npg = num_seqs * mp
        if page_table is None:
            page_table = torch.arange(npg, dtype=torch.int32).reshape(num_seqs, mp)
        page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
        npg = max(npg, int(page_table.max().item()) + 1) if page_table.numel() else npg
        codes = torch.zeros((npg, PAGE, d // 2), dtype=torch.uint8, device=device)
        scales = torch.zeros((npg, PAGE, d // 16), dtype=torch.uint8, device=device)
        idx_k = idx_k8 = idx_k8_scale = None
        if d_ik and idx_k_fp8:
            idx_k8 = torch.zeros((npg, PAGE, d_ik), dtype=torch.uint8, device=device)
            idx_k8_scale = torch.zeros((npg, PAGE), dtype=torch.float32, device=device)
        elif d_ik:
            idx_k = torch.zeros((npg, PAGE, d_ik), dtype=torch.bfloat16, device=device)
        return PagedCache(codes, scales, idx_k, page_table, idx_k8, idx_k8_scale)

    def c_struct(self, ptr=None):
        """The C struct; ptr as _pointers gives it (by default: every plane on the codes' device)."""
        ptr = ptr or _pointers(self.codes.device)
        for t, n in [(self.codes, "codes"), (self.scales, "scales"), (self.idx_k8, "idx_k8")]:
            _expect(t, _U8, n)
        _expect(self.idx_k, _B16, "idx_k")
        _expect(self.idx_k8_scale, _F32, "idx_k8_scale")
        _expect(self.page_table, _I32, "page_table")
        fp8 = self.idx_k8 is not None
        return _lib.Cache(ptr(self.codes), ptr(self.scales), ptr(self.idx_k), ptr(self.page_table),
                          self.num_pages, PAGE, self.num_seqs, self.max_pages, self.d, self.d_ik,
                          FP8E4M3 if fp8 else BF16, ptr(self.idx_k8), ptr(self.idx_k8_scale))


class Workspace:
    """Grow-only device scratch buffer handed to the library calls.  Calls that may run at the same time (on two
    streams, or in two graphs that are replayed side by side) need one each.  Threads may share one on one stream: a call
    holds its lock until all of its kernels are launched."""

    def __init__(self, device="cuda"):
        self.device = device
        self.lock = threading.RLock()
        self.buf = torch.empty(0, dtype=torch.uint8, device=device)
        self.captured = False              # a graph holds its address
        self.outgrown = []                 # buffers whose addresses graphs hold

    def get(self, nbytes):
        if torch.cuda.is_current_stream_capturing():
            if self.buf.numel() < nbytes:
                raise RuntimeError("workspace must be sized before CUDA graph capture")
            self.captured = True
        elif self.buf.numel() < nbytes:
            if self.captured:
                self.outgrown.append(self.buf)
                self.captured = False
            self.buf = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=self.device)
        return self.buf


_default_ws = {}


def _ws(ws, device):
    if ws is not None:
        return ws
    key = str(device)
    return _default_ws.get(key) or _default_ws.setdefault(key, Workspace(device))


def _call(fn, args, ws, device):
    """Call fn, which takes a workspace, on the current stream of this device, with the device current."""
    dev = device.index
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return _call(fn, args, ws, device)
    L = _lib.lib()
    need = ctypes.c_size_t(0)
    _lib.check(getattr(L, fn + "_workspace")(ctypes.byref(args), ctypes.byref(need)))
    ws = _ws(ws, device)
    with ws.lock:
        buf = ws.get(need.value)
        _on_device(buf, dev, "ws")
        _lib.check(getattr(L, fn)(ctypes.byref(args), ctypes.c_void_p(buf.data_ptr()), need.value, _stream(dev)))


def compress_quant(cache: PagedCache, seq, entry, *, m=1, C=None, Z=None, H=None, W_kv=None, W_z=None,
                   pos=None, rope_cos=None, rope_sin=None, W_ik=None, y_out=None, ws=None):
    """Compress m-token groups into FP4 Main KV entries written through the page table.
    Given mode: C (and Z when m > 1) float32 [T, d].  Projection mode: H [T, d_model]
    (bf16 or float32) with W_kv, W_z bf16 [d_model, d].  seq/entry/pos: int32 [T/m]."""
    if W_kv is not None:
        T, d_model = H.shape
        _expect(H, _B16 + _F32, "H")
        h_dtype = F32 if H.dtype == torch.float32 else BF16
    else:
        T, d_model, h_dtype = C.shape[0], 0, BF16
        _expect(C, _F32, "C")
        _expect(Z, _F32, "Z")
    for t, n in [(seq, "seq"), (entry, "entry"), (pos, "pos")]:
        _expect(t, _I32, n)
    d_rope = 0 if rope_cos is None else rope_cos.shape[1] * 2
    ptr = _pointers(cache.codes.device)
    a = _lib.CompressArgs()
    a.struct_size = ctypes.sizeof(_lib.CompressArgs)
    a.T, a.m, a.d_model, a.h_dtype = T, m, d_model, h_dtype
    a.H, a.W_kv, a.W_z, a.C, a.Z = ptr(H), ptr(W_kv), ptr(W_z), ptr(C), ptr(Z)
    a.d_rope = d_rope
    a.rope_max_pos = rope_cos.shape[0] if rope_cos is not None else 0
    a.rope_cos, a.rope_sin, a.pos = ptr(rope_cos), ptr(rope_sin), ptr(pos)
    a.seq, a.entry, a.W_ik = ptr(seq), ptr(entry), ptr(W_ik)
    a.cache = cache.c_struct(ptr)
    a.y_out = ptr(y_out)
    _call("csa2_compress_quant", a, ws, cache.codes.device)


def compress_append(cache: PagedCache, H, seq, tok_pos, W_kv, *, m=1, W_z=None, pend=None, rope_cos=None,
                    rope_sin=None, W_ik=None, y_out=None, ws=None):
    """The decode-time append: H [B, d_model] (bf16 or float32) holds one new token of each
    of B distinct sequences seq[b] at position tok_pos[b].  At m > 1 a token that does not
    complete its group waits in pend (float32 [num_seqs, 2, m, d], kept by the caller
    between calls); the completing token writes entry tok_pos // m."""
    B, d_model = H.shape
    _expect(H, _B16 + _F32, "H")
    _expect(pend, _F32, "pend")
    for t, n in [(seq, "seq"), (tok_pos, "tok_pos")]:
        _expect(t, _I32, n)
    ptr = _pointers(cache.codes.device)
    a = _lib.AppendArgs()
    a.struct_size = ctypes.sizeof(_lib.AppendArgs)
    a.B, a.m, a.d_model = B, m, d_model
    a.h_dtype = F32 if H.dtype == torch.float32 else BF16
    a.H, a.W_kv, a.W_z = ptr(H), ptr(W_kv), ptr(W_z)
    a.d_rope = 0 if rope_cos is None else rope_cos.shape[1] * 2
    a.rope_max_pos = rope_cos.shape[0] if rope_cos is not None else 0
    a.rope_cos, a.rope_sin = ptr(rope_cos), ptr(rope_sin)
    a.seq, a.tok_pos, a.pend, a.W_ik = ptr(seq), ptr(tok_pos), ptr(pend), ptr(W_ik)
    a.cache = cache.c_struct(ptr)
    a.y_out = ptr(y_out)
    _call("csa2_compress_append", a, ws, cache.codes.device)


def index_full(cache: PagedCache, q_idx, w, seq_of, n_vis, max_n, num_blocks=2048, per_block=8, k=512,
               relu=True, out=None, ws=None, group=1):
    """Full-mode indexer.  q_idx bf16 [B, H_i, d_ik], w float32 [B, H_i], seq_of / n_vis
    int32 [B].  group > 1: queries g*group .. g*group+group-1 share one sequence, whose
    indexer-K rows are read once for all of them (tensor-core scoring when group x H_i >= 16
    and the shape allows it; see include/csa2.h).  Returns (pool [B, NB*P], pool_len [B],
    topk [B, k], topk_len [B])."""
    B, H_i, _ = q_idx.shape
    dev = q_idx.device
    if out is None:
        out = (torch.empty((B, num_blocks * per_block), dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty((B, k), dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.int32, device=dev))
    pool, pool_len, topk, topk_len = out
    _expect(q_idx, _B16, "q_idx")
    _expect(w, _F32, "w")
    ptr = _pointers(dev)
    a = _lib.IndexFullArgs()
    a.struct_size = ctypes.sizeof(_lib.IndexFullArgs)
    a.B, a.H_i = B, H_i
    a.q_idx, a.w = ptr(q_idx), ptr(w)
    a.cache = cache.c_struct(ptr)
    a.seq_of, a.n_vis, a.max_n = ptr(seq_of), ptr(n_vis), int(max_n)
    a.num_blocks, a.per_block, a.k, a.relu = num_blocks, per_block, k, int(bool(relu))
    a.pool, a.pool_len, a.topk, a.topk_len = ptr(pool), ptr(pool_len), ptr(topk), ptr(topk_len)
    a.group = int(group)
    _call("csa2_index_full", a, ws, dev)
    return out


def index_reindex(cache: PagedCache, q_idx, w, seq_of, pool, pool_len, k=512, relu=True, out=None, ws=None):
    """Reindex mode: re-score only the pool.  Returns (topk [B, k], topk_len [B])."""
    B, H_i, _ = q_idx.shape
    dev = q_idx.device
    if out is None:
        out = (torch.empty((B, k), dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev))
    topk, topk_len = out
    ptr = _pointers(dev)
    a = _lib.IndexReindexArgs()
    a.struct_size = ctypes.sizeof(_lib.IndexReindexArgs)
    a.B, a.H_i = B, H_i
    a.q_idx, a.w = ptr(q_idx), ptr(w)
    a.cache = cache.c_struct(ptr)
    a.seq_of, a.pool, a.pool_len, a.pool_stride = ptr(seq_of), ptr(pool), ptr(pool_len), pool.shape[1]
    a.k, a.relu = k, int(bool(relu))
    a.topk, a.topk_len = ptr(topk), ptr(topk_len)
    _call("csa2_index_reindex", a, ws, dev)
    return out


def sparse_attn(cache: PagedCache, q, seq_of, topk, topk_len, swa, swa_scale, swa_start, swa_len, swa_max,
                softmax_scale=None, out_dtype=torch.bfloat16, out=None, lse=None, ws=None, inputs_ready=False):
    """One softmax over the selected FP4 entries plus the SWA window.  q bf16 [B, Hq, d].
    inputs_ready: the kernel launched just before on the stream writes none of this call's
    inputs (a Reuse layer after the previous layer's attention), so the call may read them
    before that kernel completes.  Returns (out [B, Hq, d], lse float32 [B, Hq])."""
    B, Hq, d = q.shape
    dev = q.device
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    _expect(q, _B16, "q")
    ptr = _pointers(dev)
    a = _lib.AttnArgs()
    a.struct_size = ctypes.sizeof(_lib.AttnArgs)
    a.B, a.Hq, a.q = B, Hq, ptr(q)
    a.cache = cache.c_struct(ptr)
    a.seq_of, a.topk, a.topk_len, a.k = ptr(seq_of), ptr(topk), ptr(topk_len), topk.shape[1]
    a.swa, a.swa_scale = ptr(swa), ptr(swa_scale)
    a.swa_rows = swa.shape[0] if swa is not None else 0
    a.swa_start, a.swa_len, a.swa_max = ptr(swa_start), ptr(swa_len), int(swa_max)
    a.softmax_scale = float(softmax_scale)
    a.out = ptr(out)
    a.out_dtype = F32 if out.dtype == torch.float32 else BF16
    a.lse = ptr(lse)
    a.inputs_ready = int(bool(inputs_ready))
    _call("csa2_sparse_attn", a, ws, dev)
    return out, lse


def swa_quant(x, swa, swa_scale, row_idx=None):
    """FP8 window rows (a bounded replay's rebuilt SWA window): each row of x (bf16 or
    float32 [R, d]) becomes E4M3 bytes with one float32 scale amax/448, written to
    swa[row_idx[r]] / swa_scale[row_idx[r]] (row r when row_idx is None)."""
    R, d = x.shape
    _expect(x, _B16 + _F32, "x")
    _expect(swa, _U8, "swa")
    _expect(swa_scale, _F32, "swa_scale")
    _expect(row_idx, _I32, "row_idx")
    ptr = _pointers(x.device)
    a = _lib.SwaQuantArgs()
    a.struct_size = ctypes.sizeof(_lib.SwaQuantArgs)
    a.R, a.d = R, d
    a.x_dtype = F32 if x.dtype == torch.float32 else BF16
    a.x, a.row_idx, a.swa, a.swa_scale = ptr(x), ptr(row_idx), ptr(swa), ptr(swa_scale)
    a.swa_rows = swa.shape[0]
    _launch("csa2_swa_quant", ctypes.byref(a), x.get_device())


_FLOAT = {torch.bfloat16: BF16, torch.float32: F32}


def _float_type(t, name):
    k = _FLOAT.get(t.dtype)
    if k is None:
        raise TypeError(f"{name}: dtype {t.dtype} is neither bfloat16 nor float32")
    return k


def _rows_of(t, dev, name):
    """(data pointer, row stride) of a matrix on CUDA device number dev whose rows are contiguous."""
    if t.get_device() != dev:                           # in line: a call of 5 us asks it five times
        _on_device(t, dev, name)
    rows, last = t.stride()
    if last != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), rows


def _dense(t, dev, dtype, name):
    """Data pointer of a contiguous tensor of one type on CUDA device number dev, 0 of None."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype} is not {dtype}")
    if t.get_device() != dev:
        _on_device(t, dev, name)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


# The argument structs of the row operators as one packed string each: a call of a single token
# costs more in ctypes field assignments than on the GPU.  0P pads a struct to its alignment.
_FP4_ROWS = "PPPii"
_RMS_NORM = struct.Struct("@NiiPiiqPPqqPifiiPqP" + _FP4_ROWS + "0P")
_ROPE = struct.Struct("@NiiiiiiiiPPqqqqPPPi0P")
_FP4_QUANT = struct.Struct("@NPiq" + _FP4_ROWS + "0P")
_FP4_LINEAR = struct.Struct("@N" + 2 * _FP4_ROWS + "Pi0P")


def _launch(fn, packed, dev):
    """Call fn on the current stream of CUDA device number dev, with that device current.  dev < 0: the operands,
    which were compared with it, are not on a GPU."""
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    call = getattr(_lib.lib(), fn)
    if _is_current(dev):
        status = call(packed, _stream(dev))
    else:
        with torch.cuda.device(dev):
            status = call(packed, _stream(dev))
    if status:
        _lib.check(status)


@dataclass
class Fp4Rows:
    """A matrix [rows, cols] in FP4: codes uint8 [rows, cols/2] (two E2M1 codes a byte, the even
    column in the low half), scales uint8 [ceil(rows/128), ceil(cols/64), 512] (E4M3 bytes in the
    tiles of include/csa2.h) and an optional float32 scale of the whole matrix (one element);
    value = code * scale * gscale."""
    codes: torch.Tensor
    scales: torch.Tensor
    gscale: Optional[torch.Tensor] = None

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def cols(self):
        return self.codes.shape[1] * 2

    @staticmethod
    def allocate(rows, cols, device, gscale=None):
        if cols <= 0 or cols % 16:
            raise ValueError(f"cols must be a positive multiple of 16 (got {cols})")
        return Fp4Rows(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                       torch.empty(((rows + 127) // 128, (cols + 63) // 64, 512), dtype=torch.uint8, device=device),
                       gscale)

    def row_scales(self):
        """The scale bytes row by row: uint8 [rows, cols/16]."""
        a, b = self.scales.shape[:2]
        return self.scales.view(a, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(a * 128, b * 4)[:self.rows,
                                                                                             :self.cols // 16]

    def fields(self, dev=None):
        """(codes, scales, gscale, rows, cols) of the C struct, after its checks; dev: the CUDA device number
        that all of them must be on (by default the codes')."""
        if dev is None:
            dev = self.codes.get_device()
        rows, half = self.codes.shape
        if self.scales.shape != ((rows + 127) // 128, (half + 31) // 32, 512):
            raise ValueError(f"scales {tuple(self.scales.shape)} do not belong to codes {tuple(self.codes.shape)}")
        g = self.gscale
        if g is not None and g.numel() != 1:
            raise ValueError("gscale must have one element")
        if dev < 0:
            raise ValueError("codes: expected a CUDA tensor")
        return (_dense(self.codes, dev, torch.uint8, "codes"), _dense(self.scales, dev, torch.uint8, "scales"),
                _dense(g, dev, torch.float32, "gscale"), rows, 2 * half)


def _norm(x, dev, weight, eps, residual, residual_out, out_form, group, out, out_stride, out_scale, out4):
    """One csa2_rms_norm call; returns residual_out (allocated here if need be)."""
    T, D = shape = x.shape
    xp, xs = _rows_of(x, dev, "x")
    wp = wt = rp = rs = op = os_ = rt = 0
    if weight is not None:
        if weight.shape != (D,):
            raise ValueError(f"weight must have {D} elements")
        wt = _float_type(weight, "weight")
        wp = _dense(weight, dev, weight.dtype, "weight")
    if residual is not None:
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=residual.dtype, device=x.device)
        elif residual_out.shape != shape or residual_out.dtype is not residual.dtype:
            raise ValueError("residual and residual_out must have x's shape and one type")
        if residual.shape != shape:
            raise ValueError("residual and residual_out must have x's shape and one type")
        rt = _float_type(residual, "residual")
        rp, rs = _rows_of(residual, dev, "residual")
        op, os_ = _rows_of(residual_out, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    _launch("csa2_rms_norm", _RMS_NORM.pack(
        _RMS_NORM.size, T, D, xp, _float_type(x, "x"), rt, xs, rp, op, rs, os_, wp, wt, eps, out_form, group, out,
        out_stride, out_scale, *out4), dev)
    return residual_out


_NO_FP4 = (0, 0, 0, 0, 0)


def rms_norm(x, weight=None, *, eps=1e-6, residual=None, residual_out=None, out_dtype=torch.bfloat16, out=None):
    """Residual addition and root-mean-square norm: h = x + residual (kept in residual_out),
    y = h / sqrt(mean(h^2) + eps) * weight.  x, residual [T, D] bf16 or float32 (rows may be
    strided); residual_out may be residual itself.  Returns (y [T, D] bf16 or float32,
    residual_out or None)."""
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    dev = x.get_device()
    return out, _norm(x, dev, weight, eps, residual, residual_out, _float_type(out, "out"), 0,
                      *_rows_of(out, dev, "out"), 0, _NO_FP4)


def rms_norm_fp8(x, weight=None, *, eps=1e-6, residual=None, residual_out=None, group=0, out=None, out_scale=None):
    """rms_norm with an E4M3 output and one float32 scale (amax / 448) for each row, or for each
    128 channels of it (group=128).  Returns (out uint8 [T, D], out_scale float32 [T, 1 or
    ceil(D/128)], residual_out or None)."""
    T, D = x.shape
    n = (D + group - 1) // group if group else 1
    if out is None:
        out = torch.empty((T, D), dtype=torch.uint8, device=x.device)
    elif out.dtype is not torch.uint8 or out.shape != x.shape:
        raise ValueError("out must be uint8 with x's shape")
    if out_scale is None:
        out_scale = torch.empty((T, n), dtype=torch.float32, device=x.device)
    elif out_scale.shape != (T, n):
        raise ValueError(f"out_scale must be [{T}, {n}]")
    dev = x.get_device()
    residual_out = _norm(x, dev, weight, eps, residual, residual_out, FP8E4M3, group, *_rows_of(out, dev, "out"),
                         _dense(out_scale, dev, torch.float32, "out_scale"), _NO_FP4)
    return out, out_scale, residual_out


def rms_norm_fp4(x, weight=None, *, eps=1e-6, residual=None, residual_out=None, gscale=None, out=None):
    """rms_norm with its output as FP4 rows (D % 16 == 0), as fp4_quant of y would give them.
    Returns (Fp4Rows, residual_out or None)."""
    if out is None:
        out = Fp4Rows.allocate(x.shape[0], x.shape[1], x.device, gscale)
    elif gscale is not None:
        raise ValueError("give gscale with out, or out alone")
    dev = x.get_device()
    return out, _norm(x, dev, weight, eps, residual, residual_out, FP4E2M1X2, 0, 0, 0, 0, out.fields(dev))


ROPE_SCALING = {"none": 0, "linear": 1, "yarn": 2}


def rope_table(positions, d_rope, *, theta=10000.0, scaling="none", factor=1.0, orig_positions=0, beta_fast=32.0,
               beta_slow=1.0, magnitude=1.0, device="cuda", out=None):
    """The rotary tables of positions [0, positions): (cos, sin), each float32 [positions,
    d_rope/2], read by rope, compress_quant and compress_append.  scaling: "none", "linear"
    (every frequency divided by factor) or "yarn" (blended by how often a channel turns within
    orig_positions).  magnitude multiplies both tables."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    shape = (max(0, positions), max(0, d_rope // 2))
    if out is None:
        out = (torch.empty(shape, dtype=torch.float32, device=device),
               torch.empty(shape, dtype=torch.float32, device=device))
    elif out[0].shape != shape or out[1].shape != shape:
        raise ValueError(f"out tables must be {list(shape)}")
    dev = out[0].get_device()
    cos, sin = (_dense(t, dev, torch.float32, "table") for t in out)
    a = _lib.RopeTableArgs(ctypes.sizeof(_lib.RopeTableArgs), positions, d_rope, ROPE_SCALING[scaling],
                           orig_positions, theta, factor, beta_fast, beta_slow, magnitude, cos, sin)
    _launch("csa2_rope_table", ctypes.byref(a), dev)
    return out


def rope(x, pos, cos, sin, *, interleaved=True, inverse=False, first=None, out=None):
    """Rotary positions: the d_rope = 2 * cos.shape[1] channels of x [T, H, D] (bf16 or float32,
    tokens and heads may be strided) from channel `first` on (by default the last d_rope, as in
    the compressor) turn by the angles of pos int32 [T]; the others are copied.  Pairs (2i, 2i+1),
    or (i, i + d_rope/2) with interleaved=False.  inverse turns back.  out=x works in place.
    Returns out."""
    T, H, D = x.shape
    positions, half = cos.shape
    if sin.shape != cos.shape or pos.shape != (T,):
        raise ValueError("cos and sin must be [positions, d_rope/2] and pos [T]")
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype is not x.dtype:
        raise ValueError("out must have x's shape and type")
    dev = x.get_device()
    if out.get_device() != dev:
        _on_device(out, dev, "out")
    xt, xh, xc = x.stride()
    ot, oh, oc = out.stride()
    if (xc != 1 or oc != 1) and D > 1:
        raise ValueError("the last dimension must be contiguous")
    _launch("csa2_rope", _ROPE.pack(
        _ROPE.size, T, H, D, 2 * half, D - 2 * half if first is None else first, 1 if interleaved else 0,
        1 if inverse else 0, _float_type(x, "x"), x.data_ptr(), out.data_ptr(), xt, xh, ot, oh,
        _dense(pos, dev, torch.int32, "pos"), _dense(cos, dev, torch.float32, "cos"),
        _dense(sin, dev, torch.float32, "sin"), positions), dev)
    return out


def fp4_quant(x, gscale=None, out=None):
    """Rows x [T, K] (bf16 or float32, rows may be strided, K % 16 == 0) to FP4 rows: x / gscale
    with one E4M3 scale per 16 columns.  Returns Fp4Rows."""
    T, K = x.shape
    if out is None:
        out = Fp4Rows.allocate(T, K, x.device, gscale)
    elif gscale is not None:
        raise ValueError("give gscale with out, or out alone")
    dev = x.get_device()
    xp, xs = _rows_of(x, dev, "x")
    fields = out.fields(dev)
    if fields[3] != T or fields[4] != K:
        raise ValueError("out must have x's shape")
    _launch("csa2_fp4_quant", _FP4_QUANT.pack(_FP4_QUANT.size, xp, _float_type(x, "x"), xs, *fields), dev)
    return out


def fp4_linear(x: Fp4Rows, w: Fp4Rows, *, out_dtype=torch.bfloat16, out=None):
    """The product of FP4 rows x [T, K] with FP4 weights w [N, K] (K % 32 == 0) on the
    block-scaled tensor cores.  Returns out [T, N] bf16 or float32."""
    dev = x.codes.get_device()
    fx, fw = x.fields(dev), w.fields(dev)
    if out is None:
        out = torch.empty((fx[3], fw[3]), dtype=out_dtype, device=x.codes.device)
    elif out.shape != (fx[3], fw[3]):
        raise ValueError(f"out must be [{fx[3]}, {fw[3]}]")
    _launch("csa2_fp4_linear", _FP4_LINEAR.pack(_FP4_LINEAR.size, *fx, *fw, _dense(out, dev, out.dtype, "out"),
                                                _float_type(out, "out")), dev)
    return out


# ---- the paged 8-bit cache --------------------------------------------------------------------

_KV8_CACHE = "PPPPPPPiiiiii"
_PAGE_PLAN = struct.Struct("@NiiiiPPPPPPPPPPP")
_KV8_APPEND = struct.Struct("@NiiiPPqqqqPP" + _KV8_CACHE + "0P")
_KV8_SELECT = struct.Struct("@NiiiiiiiPqqPP" + _KV8_CACHE + "0P" + "PP")
_KV8_ATTN = struct.Struct("@NiiiiifPqqPP" + _KV8_CACHE + "0P" + "PiPiP")


@dataclass
class Kv8Cache:
    """Paged keys and values in 8 bits for grouped-query attention layers: k, v uint8 (E4M3 bytes)
    [pages, Hkv, 64, D], k_scale, v_scale float32 [pages, Hkv], page_table int32 [seqs, max_pages], and, if
    kv8_select is to choose pages, their summaries mean int8 [pages, Hkv, D] with mean_scale float32
    [pages, Hkv]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    page_table: torch.Tensor
    mean: Optional[torch.Tensor] = None
    mean_scale: Optional[torch.Tensor] = None

    @staticmethod
    def allocate(num_pages, heads, D, page_table, mean=True):
        """A cache of num_pages pages on the page table's device."""
        new = lambda dtype, *s: torch.zeros((num_pages, heads) + s, dtype=dtype, device=page_table.device)
        return Kv8Cache(new(torch.uint8, PAGE, D), new(torch.uint8, PAGE, D), new(torch.float32), new(torch.float32),
                        page_table, new(torch.int8, D) if mean else None, new(torch.float32) if mean else None)

    def fields(self, dev):
        """The C struct's values, after its checks; dev: the CUDA device number that all planes must be on."""
        k, v, ks, vs, table, m, ms = self.k, self.v, self.k_scale, self.v_scale, self.page_table, self.mean, self.mean_scale
        shape = k.shape
        pages, heads, slots, D = shape
        per = (pages, heads)
        if slots != PAGE or v.shape != shape:
            raise ValueError(f"k and v must be [pages, heads, {PAGE}, D] alike")
        if ks.shape != per or vs.shape != per:
            raise ValueError(f"k_scale and v_scale must be [{pages}, {heads}]")
        if (m is None) != (ms is None):
            raise ValueError("mean and mean_scale go together")
        if m is not None and (m.shape != (pages, heads, D) or ms.shape != per):
            raise ValueError(f"mean must be [{pages}, {heads}, {D}] and mean_scale [{pages}, {heads}]")
        at = []
        for t, dtype, name in zip((k, v, ks, vs, m, ms, table), _KV8_TYPES, _KV8_NAMES):
            if t is None:
                at.append(0)
                continue
            if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
                _dense(t, dev, dtype, name)              # says which
            at.append(t.data_ptr())
        seqs, most = table.shape
        return (*at, pages, PAGE, seqs, most, heads, D)


_KV8_TYPES = (torch.uint8, torch.uint8, torch.float32, torch.float32, torch.int8, torch.float32, torch.int32)
_KV8_NAMES = ("k plane", "v plane", "k_scale", "v_scale", "mean", "mean_scale", "page_table")
_ws_of = {}                                # the default workspaces by device number and stream


def _stream_ws(dev, stream, device):
    return _ws_of.get((dev, stream)) or _ws_of.setdefault((dev, stream), Workspace(device))


def _launch_ws(fn, packed, ws, device, dev):
    """_launch of a call that takes a workspace (ws None: the stream's own, or, in a capture, the graph's).  It is offered
    the one there is, and asked what it needs only if that is too small."""
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return _launch_ws(fn, packed, ws, device, dev)
    L = _lib.lib()
    stream, call = _stream(dev), getattr(L, fn)
    need = ctypes.c_size_t(0)
    if ws is None and torch.cuda.is_current_stream_capturing():
        # memory of the graph's own: graphs share no workspace, and none with eager calls
        _lib.check(getattr(L, fn + "_workspace")(packed, ctypes.byref(need)))
        buf = torch.empty(need.value, dtype=torch.uint8, device=device)
        _lib.check(call(packed, buf.data_ptr(), need.value, stream))
        return
    if ws is None:
        ws = _stream_ws(dev, stream, device)
    with ws.lock:                              # one call's kernels behind another's, not in between
        buf = ws.get(0)
        if buf.get_device() != dev:
            _on_device(buf, dev, "ws")
        status = call(packed, buf.data_ptr(), buf.numel(), stream)
        if status == _TOO_SMALL:
            _lib.check(getattr(L, fn + "_workspace")(packed, ctypes.byref(need)))
            buf = ws.get(need.value)
            status = call(packed, buf.data_ptr(), need.value, stream)
        if status:
            _lib.check(status)


_TOO_SMALL = 3                             # CSA2_ERR_WORKSPACE_TOO_SMALL


def _heads_of(t, dev, name):
    """(data pointer, token stride, head stride) of a [T, H, D] tensor with contiguous channels."""
    if t.get_device() != dev:
        _on_device(t, dev, name)
    st, sh, sc = t.stride()
    if sc != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), st, sh


def _step(cache, start, length, dev):
    """(sequences, start, length) of a step's rows."""
    S, = length.shape
    if start.shape != (S + 1,) or S > cache.page_table.shape[0]:
        raise ValueError("start must be [S + 1] and length [S], S at most the page table's rows")
    return S, *_i32_at(dev, (start, length), ("start", "length"))


def _i32_at(dev, tensors, names):
    """Addresses of contiguous int32 tensors on CUDA device number dev."""
    at = []
    for t, name in zip(tensors, names):
        if t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous():
            _dense(t, dev, torch.int32, name)            # says which
        at.append(t.data_ptr())
    return at


@dataclass
class PagePlan:
    """The tables of a step (page_plan): start int32 [S+1], seq, pos, slot int32 [tokens], length int32 [S] and
    head int32 [1] after it."""
    start: torch.Tensor
    seq: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor
    length: torch.Tensor
    head: torch.Tensor

    @staticmethod
    def allocate(seqs, tokens, device):
        rows = torch.empty(3 * tokens + 2 * seqs + 2, dtype=torch.int32, device=device)
        seq, pos, slot, start, length, head = torch.unsafe_split_with_sizes(
            rows, (tokens, tokens, tokens, seqs + 1, seqs, 1))       # one allocation: six take twice as long
        return PagePlan(start, seq, pos, slot, length, head)


def page_plan(length, add, page_table, free_pages, free_head, tokens, *, out=None):
    """The tables of a step in which sequence s, holding length[s] tokens, gets add[s] more (int32 [S]): where its rows
    stand (start), each row's sequence, position and slot (-1 past the last row, of `tokens`), and page_table
    int32 [S, max_pages] extended by pages off free_pages int32 [F] from free_head int32 [1] on.
    out may hold length and free_head themselves, which then advance.  Returns PagePlan."""
    S, = length.shape
    if add.shape != (S,) or page_table.shape[0] != S or free_head.numel() != 1:
        raise ValueError("length and add must be [S], page_table [S, max_pages], free_head [1]")
    dev = length.get_device()
    ins = _i32_at(dev, (length, add, free_pages, free_head, page_table), ("length", "add", "free_pages", "free_head", "page_table"))
    if out is None:
        out = PagePlan.allocate(S, tokens, length.device)
        at = out.start.data_ptr()                      # one allocation: seq, pos, slot, start, length, head
        outs = (at, at - 12 * tokens, at - 8 * tokens, at - 4 * tokens, at + 4 * S + 4, at + 8 * S + 4)
    else:
        if (out.start.shape != (S + 1,) or out.length.shape != (S,) or out.head.numel() != 1
                or any(t.shape != (tokens,) for t in (out.seq, out.pos, out.slot))):
            raise ValueError("out must be PagePlan.allocate(S, tokens)")
        outs = _i32_at(dev, (out.start, out.seq, out.pos, out.slot, out.length, out.head),
                       ("start", "seq", "pos", "slot", "out.length", "out.head"))
    _launch("csa2_page_plan", _PAGE_PLAN.pack(_PAGE_PLAN.size, S, page_table.shape[1], tokens, free_pages.shape[0], *ins, *outs), dev)
    return out


def kv8_append(cache: Kv8Cache, k, v, start, length):
    """Quantise the new keys and values k, v [T, Hkv, D] (bf16 or float32; tokens and heads may be strided)
    into the cache: sequence s's are rows start[s] .. start[s+1]-1, and it holds length[s] tokens with them (int32,
    as page_plan returns them)."""
    T, H, D = k.shape
    if v.shape != k.shape or (H, D) != (cache.k.shape[1], cache.k.shape[3]):
        raise ValueError("k and v must be [T, Hkv, D] of the cache's heads and channels")
    if v.dtype is not k.dtype:
        raise TypeError("k and v must have one type")
    dev = k.get_device()
    kp, kt, kh = _heads_of(k, dev, "k")
    vp, vt, vh = _heads_of(v, dev, "v")
    S, sp, lp = _step(cache, start, length, dev)
    _launch("csa2_kv8_append", _KV8_APPEND.pack(_KV8_APPEND.size, T, S, _float_type(k, "k"), kp, vp, kt, kh, vt, vh, sp, lp,
                                                *cache.fields(dev)), dev)


def kv8_select(cache: Kv8Cache, q, start, length, k, *, first=1, recent=1, max_length=None, out=None, ws=None):
    """The pages each new token attends to, by key head: the `first` oldest, the `recent` newest and the best-scoring
    others, k at most.  q bf16 [T, Hq, D] (tokens and heads may be strided); start, length as in
    kv8_append; max_length: a bound of length.  It sizes the workspace and picks the kernel; by default it is the page table's
    width, which costs where that is much wider than the contexts (2048 rows at 32K: 77 us with the bound, 480 under a table
    for a million tokens).  Returns (pages int32 [T, Hkv, k], ascending and padded with -1, count int32 [T, Hkv])."""
    T, Hq, D = q.shape
    H = cache.k.shape[1]
    _expect(q, _B16, "q")
    if D != cache.k.shape[3]:
        raise ValueError("q must have the cache's channels")
    if out is None:
        out = (torch.empty((T, H, k), dtype=torch.int32, device=q.device),
               torch.empty((T, H), dtype=torch.int32, device=q.device))
    elif out[0].shape != (T, H, k) or out[1].shape != (T, H):
        raise ValueError(f"out must be int32 [{T}, {H}, {k}] and [{T}, {H}]")
    dev = q.get_device()
    qp, qt, qh = _heads_of(q, dev, "q")
    S, sp, lp = _step(cache, start, length, dev)
    if max_length is None:
        max_length = min(cache.page_table.shape[1] * PAGE, 1 << 21)
    _launch_ws("csa2_kv8_select", _KV8_SELECT.pack(
        _KV8_SELECT.size, T, S, Hq, k, first, recent, max_length, qp, qt, qh, sp, lp, *cache.fields(dev),
        _dense(out[0], dev, torch.int32, "pages"), _dense(out[1], dev, torch.int32, "count")), ws, q.device, dev)
    return out


def kv8_attn(cache: Kv8Cache, q, start, length, *, max_new=None, pages=None, window=0, softmax_scale=None,
             out_dtype=torch.bfloat16, out=None, lse=None, ws=None):
    """Causal attention of the new tokens q bf16 [T, Hq, D] (tokens and heads may be strided) over the cache, which
    holds their keys and values already; start, length as in kv8_append.  max_new: about how many new tokens a sequence
    has at most.  It picks one kernel for all sequences of the call; by default it is T - S + 1, which one has if all have
    some, and which rows of padding raise: give it for a padded step.  Single rows beside a long chunk are faster in a call
    of their own, over their range of the page table's rows, of start and of length.  pages int32 [T, Hkv, n]: only these
    pages (kv8_select).  window: only so many newest positions.  Returns (out [T, Hq, D] bf16 or float32, lse float32
    [T, Hq])."""
    T, Hq, D = q.shape
    H = cache.k.shape[1]
    _expect(q, _B16, "q")
    if D != cache.k.shape[3]:
        raise ValueError("q must have the cache's channels")
    dev = q.get_device()
    if out is None:
        out = torch.empty((T, Hq, D), dtype=out_dtype, device=q.device)
        op = out.data_ptr()
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    else:
        op = _dense(out, dev, out.dtype, "out")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
        lp = lse.data_ptr()
    elif lse.shape != (T, Hq):
        raise ValueError(f"lse must be [{T}, {Hq}]")
    else:
        lp = _dense(lse, dev, torch.float32, "lse")
    n = 0
    if pages is not None:
        if pages.shape[:2] != (T, H) or len(pages.shape) != 3:
            raise ValueError(f"pages must be [{T}, {H}, n]")
        n = pages.shape[2]
        if n == 0:                             # (its address is 0, which would mean all pages)
            raise ValueError("pages must have room for at least one page; -1 for none")
    qp, qt, qh = _heads_of(q, dev, "q")
    S, sp, lengths = _step(cache, start, length, dev)
    _launch_ws("csa2_kv8_attn", _KV8_ATTN.pack(
        _KV8_ATTN.size, T, S, Hq, max(T - S, 0) + 1 if max_new is None else max_new, window,
        1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale, qp, qt, qh, sp, lengths, *cache.fields(dev),
        _dense(pages, dev, torch.int32, "pages"), n, op, _float_type(out, "out"), lp), ws, q.device, dev)
    return out, lse


def device_error():
    """Synchronise and return (and clear) the device error word (a non-zero word is
    returned, not raised: the library reports it as CSA2_ERR_DEVICE_CHECK / _TIMEOUT)."""
    w = ctypes.c_uint32(0)
    st = _lib.lib().csa2_get_device_error(ctypes.byref(w))
    if st not in (0, 5, 6):
        _lib.check(st)
    return w.value


def version():
    return _lib.lib().csa2_version()


def selftest_wait_timeout(polls=1000):
    """Run the bounded-wait failure path once (one CTA waits on an mbarrier nothing
    arrives on, gives up after `polls` polls and sets the timeout bit of the device error
    word)."""
    _lib.check(_lib.lib().csa2_selftest_wait_timeout(int(polls), _stream(torch.cuda.current_device())))
