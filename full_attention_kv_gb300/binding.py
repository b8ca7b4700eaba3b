"""Thin ctypes binding of libhsa (include/hsa.h), same entry-point names.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  If libhsa.so has not been
built, every call raises; there is no fallback of any kind.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libhsa.so")

HSA_OK = 0
HSA_INVALID_ARG = 1
HSA_UNSUPPORTED_SHAPE = 2
HSA_CUDA_ERROR = 3
HSA_OUT_OF_RANGE = 4

HSA_DECODE_APPEND = 1
HSA_DECODE_EARLY_POOL_READ = 2

HSA_DEVERR_BAD_BLOCK = 1
HSA_DEVERR_BAD_PAGE = 2
HSA_DEVERR_BAD_SEQ = 4
HSA_DEVERR_BAD_RING = 8
HSA_DEVERR_BAD_LEN = 16
HSA_DEVERR_TIMEOUT = 32

# every symbol include/hsa.h declares
EXPORTS = ("hsa_kv_append", "hsa_rope", "hsa_rope_kv_append", "hsa_decode_workspace_bytes", "hsa_decode_attn",
           "hsa_decode_attn_append", "hsa_decode_attn_ex", "hsa_decode_attn_noalloc",
           "hsa_decode_shared_workspace_bytes", "hsa_decode_attn_shared",
           "hsa_decode_weights_workspace_bytes", "hsa_decode_attn_weights",
           "hsa_prefill_weights_workspace_bytes", "hsa_prefill_weights",
           "hsa_prefill_attn", "hsa_kv_select", "hsa_kv_compact",
           "hsa_swa_prefetch",
           "hsa_window_safe_len", "hsa_window_safe_len_bitmap", "hsa_status_string")
# every symbol include/hsa_tree.h declares
TREE_EXPORTS = ("hsa_ptree_create", "hsa_ptree_destroy", "hsa_ptree_match",
                "hsa_ptree_match_batch", "hsa_ptree_insert", "hsa_ptree_unlock",
                "hsa_ptree_evict_full", "hsa_ptree_evict_swa", "hsa_ptree_stats")


class HsaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))


class HsaPools(ctypes.Structure):
    """Mirror of the C struct hsa_pools."""
    _fields_ = [
        ("n_layers", ctypes.c_int32),
        ("layer_is_full", ctypes.POINTER(ctypes.c_uint8)),
        ("k", ctypes.POINTER(ctypes.c_void_p)),
        ("v", ctypes.POINTER(ctypes.c_void_p)),
        ("num_blocks", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("block_tables", ctypes.c_void_p),
        ("max_blocks", ctypes.c_int32),
        ("ring_row", ctypes.c_void_p),
        ("n_ring_rows", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("W", ctypes.c_int32),
        ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("layer_kv_fp8", ctypes.POINTER(ctypes.c_uint8)),
    ]


class HsaRopeParams(ctypes.Structure):
    """Mirror of the C struct hsa_rope_params."""
    _fields_ = [
        ("rot_dim", ctypes.c_int32),
        ("n_axes", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("inv_freq", ctypes.POINTER(ctypes.c_double)),
        ("axis_of_pair", ctypes.POINTER(ctypes.c_uint8)),
    ]


_lib = None


def lib():
    """Load libhsa.so (raises if it was not built: the CUDA path is the only path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libhsa.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        pp = ctypes.POINTER(HsaPools)
        L.hsa_kv_append.restype = ctypes.c_int
        L.hsa_kv_append.argtypes = [pp, i32, vp, vp, vp, vp, vp, i32, i32, vp, vp]
        i64 = ctypes.c_int64
        rp = ctypes.POINTER(HsaRopeParams)
        L.hsa_rope.restype = ctypes.c_int
        L.hsa_rope.argtypes = [rp, vp, i64, vp, i64, vp, i32, i32, i32, i32, vp, vp, vp]
        L.hsa_rope_kv_append.restype = ctypes.c_int
        L.hsa_rope_kv_append.argtypes = [pp, i32, rp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp,
                                         i32, i32, vp, vp, vp, vp]
        L.hsa_decode_workspace_bytes.restype = sz
        L.hsa_decode_workspace_bytes.argtypes = [pp, i32, i32]
        L.hsa_decode_attn.restype = ctypes.c_int
        L.hsa_decode_attn.argtypes = [pp, i32, vp, vp, vp, vp, i32, i32, f32, vp, vp, sz, i32,
                                      vp, vp]
        L.hsa_decode_attn_append.restype = ctypes.c_int
        L.hsa_decode_attn_append.argtypes = [pp, i32, vp, vp, vp, vp, i32, i32, f32, vp, vp, sz,
                                             i32, vp, vp]
        L.hsa_decode_attn_ex.restype = ctypes.c_int
        L.hsa_decode_attn_ex.argtypes = [pp, i32, vp, vp, vp, vp, i32, i32, f32, vp, vp, sz,
                                         i32, i32, vp, vp]
        L.hsa_decode_attn_noalloc.restype = ctypes.c_int
        L.hsa_decode_attn_noalloc.argtypes = [pp, i32, vp, vp, vp, vp, i32, i32, f32, vp, i32,
                                              vp, vp]
        L.hsa_decode_shared_workspace_bytes.restype = sz
        L.hsa_decode_shared_workspace_bytes.argtypes = [pp, i32, i32, i32]
        L.hsa_decode_attn_shared.restype = ctypes.c_int
        L.hsa_decode_attn_shared.argtypes = [pp, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, f32,
                                             vp, vp, sz, i32, i32, vp, vp]
        L.hsa_prefill_attn.restype = ctypes.c_int
        L.hsa_prefill_attn.argtypes = [pp, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, f32, vp,
                                       vp, vp]
        L.hsa_decode_weights_workspace_bytes.restype = sz
        L.hsa_decode_weights_workspace_bytes.argtypes = [pp, i32, i32, i32]
        L.hsa_decode_attn_weights.restype = ctypes.c_int
        L.hsa_decode_attn_weights.argtypes = [pp, i32, vp, vp, vp, vp, i32, i32, f32, vp, vp, f32, vp,
                                              i32, vp, sz, i32, i32, vp, vp]
        L.hsa_prefill_weights_workspace_bytes.restype = sz
        L.hsa_prefill_weights_workspace_bytes.argtypes = [pp, i32, i32]
        L.hsa_prefill_weights.restype = ctypes.c_int
        L.hsa_prefill_weights.argtypes = [pp, i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, f32, vp, i32,
                                          vp, sz, vp, vp]
        L.hsa_kv_select.restype = ctypes.c_int
        L.hsa_kv_select.argtypes = [vp, i32, i32, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        L.hsa_kv_compact.restype = ctypes.c_int
        L.hsa_kv_compact.argtypes = [pp, i32, vp, i32, i32, vp, vp, i32, vp, i32, vp, vp, i32, vp, vp]
        L.hsa_swa_prefetch.restype = ctypes.c_int
        L.hsa_swa_prefetch.argtypes = [pp, i32, vp, vp, i32, vp, vp, i32, vp, vp]
        L.hsa_window_safe_len.restype = ctypes.c_int
        L.hsa_window_safe_len.argtypes = [vp, vp, i32, i32, vp, vp]
        L.hsa_window_safe_len_bitmap.restype = ctypes.c_int
        L.hsa_window_safe_len_bitmap.argtypes = [vp, vp, vp, i32, i32, vp, vp]
        L.hsa_status_string.restype = ctypes.c_char_p
        L.hsa_status_string.argtypes = [ctypes.c_int]
        i64, pi32 = ctypes.c_int64, ctypes.POINTER(ctypes.c_int32)
        L.hsa_ptree_create.restype = ctypes.c_int
        L.hsa_ptree_create.argtypes = [i32, i32, ctypes.POINTER(vp)]
        L.hsa_ptree_destroy.restype = None
        L.hsa_ptree_destroy.argtypes = [vp]
        L.hsa_ptree_match.restype = ctypes.c_int
        L.hsa_ptree_match.argtypes = [vp, vp, i32, i32, i32, pi32, vp, pi32, vp,
                                      ctypes.POINTER(i64)]
        L.hsa_ptree_match_batch.restype = ctypes.c_int
        L.hsa_ptree_match_batch.argtypes = [vp, vp, vp, i32, vp, vp, vp]
        L.hsa_ptree_insert.restype = ctypes.c_int
        L.hsa_ptree_insert.argtypes = [vp, vp, vp, i32, i32, vp, vp, pi32, pi32]
        L.hsa_ptree_unlock.restype = ctypes.c_int
        L.hsa_ptree_unlock.argtypes = [vp, i64]
        L.hsa_ptree_evict_full.restype = ctypes.c_int
        L.hsa_ptree_evict_full.argtypes = [vp, i32, vp, i32, pi32, vp, i32, pi32]
        L.hsa_ptree_evict_swa.restype = ctypes.c_int
        L.hsa_ptree_evict_swa.argtypes = [vp, i32, vp, pi32]
        L.hsa_ptree_stats.restype = ctypes.c_int
        L.hsa_ptree_stats.argtypes = [vp, ctypes.POINTER(i64), pi32, pi32]
        _lib = L
    return _lib


def status_string(s):
    return lib().hsa_status_string(int(s)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _made(make, ref, stream):
    """make(), a tensor for a call whose kernels run on `stream`: its memory, and what fills
    it, belong to that stream, so that neither work still queued on the current stream nor
    the memory's next use there can meet the kernels.  (The current stream counts as a user
    of it, as the caller may read the result there.)"""
    if stream is None or not ref.is_cuda:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=ref.device) if int(stream) else \
            torch.cuda.default_stream(ref.device)
    here = torch.cuda.current_stream(ref.device)
    if stream.cuda_stream == here.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(here)
    return t


def _empty(shape, like, stream):
    if stream is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    return _made(lambda: torch.empty(shape, dtype=like.dtype, device=like.device), like, stream)


def _need(t, name, dtype, device=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got %d" % (name, ndim, t.dim()))


def _shape(t, name, shape):
    """The library takes plain pointers: sizes the pool implies are checked here."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _same_device(ref, *ts):
    for t in ts:
        if t is not None and t.device != ref.device:
            raise ValueError("all device tensors must be on %s" % ref.device)


def _need_err(dev_err):
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32)
        if dev_err.numel() < 1:
            raise ValueError("dev_err must hold one int32")


def _check(fn, status):
    if status != HSA_OK:
        raise HsaError(fn, status)


HSA_KV_E4M3 = 1
HSA_KV_E5M2 = 2


def fp8_code(fmt):
    """layer_kv_fp8 value of a format: False / None / 0 -> 0 (bf16), True / 1 / "e4m3"
    -> HSA_KV_E4M3, 2 / "e5m2" -> HSA_KV_E5M2."""
    if fmt is None or fmt is False or (isinstance(fmt, int) and not isinstance(fmt, bool)
                                       and fmt == 0):
        return 0
    if fmt is True or fmt == "e4m3" or (isinstance(fmt, int) and fmt == HSA_KV_E4M3):
        return HSA_KV_E4M3
    if fmt == "e5m2" or (isinstance(fmt, int) and fmt == HSA_KV_E5M2):
        return HSA_KV_E5M2
    raise ValueError("unknown FP8 format %r" % (fmt,))


class DualPool:
    """The dual KV pool of one model: the C struct plus the tensors it points at.

    Full layers own K/V tensors [num_blocks, Hkv, page, d]; sliding layers own
    rings [n_ring_rows, Hkv, W, d]; block_tables [batch, max_blocks] and ring_row
    [batch] (int32) are shared by every layer of their kind.
    """

    def __init__(self, layer_is_full, k, v, block_tables, ring_row, Hq, W=128, page=64,
                 kv_fp8=None, Hkv=None, d=None, num_blocks=None):
        """kv_fp8[l] marks an FP8 full layer (True or "e4m3": E4M3 codes; "e5m2":
        E5M2 codes; False / None: bf16): k[l], v[l] are then flat uint8 buffers of
        num_blocks * Hkv * page * (d + 4) bytes (codes, then fp32 scales;
        include/hsa.h gives the layout), and Hkv, d, num_blocks must be passed."""
        self.layer_is_full = [bool(x) for x in layer_is_full]
        self.k, self.v = list(k), list(v)
        self.block_tables, self.ring_row = block_tables, ring_row
        n = len(self.layer_is_full)
        assert len(self.k) == n and len(self.v) == n
        self.kv_fp8 = [fp8_code(x) for x in kv_fp8] if kv_fp8 is not None else [0] * n
        assert len(self.kv_fp8) == n
        _need(block_tables, "block_tables", torch.int32, ndim=2)
        _need(ring_row, "ring_row", torch.int32, ndim=1)
        n_rows = None
        for l in range(n):
            if self.kv_fp8[l]:
                if not self.layer_is_full[l]:
                    raise ValueError("layer %d: only full layers can be FP8" % l)
                if Hkv is None or d is None or num_blocks is None:
                    raise ValueError("FP8 layers need Hkv, d and num_blocks")
                for t, nm in ((self.k[l], "k"), (self.v[l], "v")):
                    _need(t, "%s[%d]" % (nm, l), torch.uint8, ndim=1)
                    if t.numel() != num_blocks * Hkv * page * (d + 4):
                        raise ValueError("%s[%d]: wrong FP8 layer size" % (nm, l))
                continue
            _need(self.k[l], "k[%d]" % l, torch.bfloat16, ndim=4)
            _need(self.v[l], "v[%d]" % l, torch.bfloat16, ndim=4)
            if self.k[l].shape != self.v[l].shape:
                raise ValueError("k[%d] and v[%d] differ in shape" % (l, l))
            nb, hk, rows, dd = self.k[l].shape
            if self.layer_is_full[l]:
                if rows != page:
                    raise ValueError("full layer %d: rows per block %d != page %d" % (l, rows, page))
                num_blocks = nb if num_blocks is None else num_blocks
                if nb != num_blocks:
                    raise ValueError("full layers disagree on num_blocks")
            else:
                if rows != W:
                    raise ValueError("sliding layer %d: ring slots %d != W %d" % (l, rows, W))
                n_rows = nb if n_rows is None else n_rows
                if nb != n_rows:
                    raise ValueError("sliding layers disagree on ring rows")
            Hkv = hk if Hkv is None else Hkv
            d = dd if d is None else d
            if hk != Hkv or dd != d:
                raise ValueError("layers disagree on Hkv / d")
        self._full = (ctypes.c_uint8 * n)(*[1 if f else 0 for f in self.layer_is_full])
        self._fp8 = (ctypes.c_uint8 * n)(*self.kv_fp8)
        self._k = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.k])
        self._v = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.v])
        self.c = HsaPools(
            n_layers=n, layer_is_full=ctypes.cast(self._full, ctypes.POINTER(ctypes.c_uint8)),
            k=ctypes.cast(self._k, ctypes.POINTER(ctypes.c_void_p)),
            v=ctypes.cast(self._v, ctypes.POINTER(ctypes.c_void_p)),
            num_blocks=num_blocks or 0, page_size=page, block_tables=block_tables.data_ptr(),
            max_blocks=block_tables.shape[1], ring_row=ring_row.data_ptr(),
            n_ring_rows=n_rows or 0, batch=block_tables.shape[0], W=W, Hq=Hq, Hkv=Hkv or 0,
            d=d or 0, layer_kv_fp8=ctypes.cast(self._fp8, ctypes.POINTER(ctypes.c_uint8)))
        self.Hq, self.Hkv, self.d, self.W, self.page = Hq, Hkv, d, W, page
        self.num_blocks = num_blocks or 0

    def fp8_views(self, layer):
        """Views of an FP8 layer: (K codes [nb, Hkv, page, d] in stored byte order,
        K scales [nb, Hkv, page] fp32, V codes [nb, Hkv, d, page] (transposed, stored
        key order), V scales [nb, Hkv, page] fp32)."""
        if not self.kv_fp8[layer]:
            raise ValueError("layer %d is not FP8" % layer)
        nb, hk, pg, dd = self.num_blocks, self.Hkv, self.page, self.d
        cb = nb * hk * pg * dd
        out = []
        for buf, shape in ((self.k[layer], (nb, hk, pg, dd)), (self.v[layer], (nb, hk, dd, pg))):
            out.append(buf[:cb].view(shape))
            out.append(buf[cb:].view(torch.float32).view(nb, hk, pg))
        return tuple(out)

    @classmethod
    def allocate(cls, layer_is_full, num_blocks, n_ring_rows, block_tables, ring_row, Hq, Hkv,
                 d=128, W=128, page=64, device="cuda", kv_fp8=False):
        """Zero-filled pools (rows past a sequence's length must hold finite values).
        kv_fp8=True / "e4m3" / "e5m2" stores every full layer as an FP8 layer of that
        format (sliding rings stay bf16)."""
        k, v = [], []
        fp8 = [fp8_code(kv_fp8) if f else 0 for f in layer_is_full]
        for f, q8 in zip(layer_is_full, fp8):
            if q8:
                nbytes = num_blocks * Hkv * page * (d + 4)
                k.append(torch.zeros(nbytes, dtype=torch.uint8, device=device))
                v.append(torch.zeros(nbytes, dtype=torch.uint8, device=device))
                continue
            shape = (num_blocks, Hkv, page, d) if f else (n_ring_rows, Hkv, W, d)
            k.append(torch.zeros(shape, dtype=torch.bfloat16, device=device))
            v.append(torch.zeros(shape, dtype=torch.bfloat16, device=device))
        return cls(layer_is_full, k, v, block_tables, ring_row, Hq, W=W, page=page, kv_fp8=fp8,
                   Hkv=Hkv, d=d, num_blocks=num_blocks)

    def ref(self):
        return ctypes.byref(self.c)


def hsa_kv_append(pool, layer, k_new, v_new, cu_tokens, seq_idx, start_pos, dev_err=None,
                  stream=None):
    _need(k_new, "k_new", torch.bfloat16, ndim=3)
    _need(v_new, "v_new", torch.bfloat16, ndim=3)
    for n, t in (("cu_tokens", cu_tokens), ("seq_idx", seq_idx), ("start_pos", start_pos)):
        _need(t, n, torch.int32, ndim=1)
    R = seq_idx.shape[0]
    if cu_tokens.shape[0] != R + 1 or start_pos.shape[0] != R:
        raise ValueError("cu_tokens must be [R+1] and start_pos [R]")
    _shape(k_new, "k_new", (k_new.shape[0], pool.Hkv, pool.d))
    _shape(v_new, "v_new", k_new.shape)
    _need_err(dev_err)
    _same_device(k_new, v_new, cu_tokens, seq_idx, start_pos, dev_err)
    s = lib().hsa_kv_append(pool.ref(), int(layer), _ptr(k_new), _ptr(v_new), _ptr(cu_tokens),
                            _ptr(seq_idx), _ptr(start_pos), R, k_new.shape[0], _ptr(dev_err),
                            _stream(stream))
    _check("hsa_kv_append", s)


class Rope:
    """Rotary positions: the C struct hsa_rope_params and the arrays it points at.

    rot_dim        the leading values of a head that are turned (a multiple of 16)
    base           inv_freq[i] = base ** (-2 i / rot_dim), unless inv_freq is given
                   (rot_dim / 2 numbers, or a tensor: any scaled frequencies)
    sections       pairs on each axis in order, e.g. (16, 24, 24) for time, height and
                   width; or axis_of_pair, the axis of each pair (any interleaving)
    interleaved    pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2)
    scale          of the turned values
    """

    def __init__(self, rot_dim=128, base=10000.0, sections=None, interleaved=False, scale=1.0,
                 inv_freq=None, axis_of_pair=None):
        half = int(rot_dim) // 2
        if inv_freq is None:
            inv_freq = [float(base) ** (-2.0 * i / rot_dim) for i in range(half)]
        elif isinstance(inv_freq, torch.Tensor):
            inv_freq = inv_freq.detach().double().cpu().tolist()
        inv_freq = [float(f) for f in inv_freq]
        if len(inv_freq) != half:
            raise ValueError("inv_freq must hold rot_dim / 2 = %d numbers, got %d"
                             % (half, len(inv_freq)))
        if sections is not None:
            if axis_of_pair is not None:
                raise ValueError("give sections or axis_of_pair, not both")
            if any(int(s) < 0 for s in sections) or sum(int(s) for s in sections) != half:
                raise ValueError("sections must add up to rot_dim / 2 = %d" % half)
            axis_of_pair = [a for a, s in enumerate(sections) for _ in range(int(s))]
            n_axes = len(sections)
        elif axis_of_pair is not None:
            if isinstance(axis_of_pair, torch.Tensor):
                axis_of_pair = axis_of_pair.cpu().tolist()
            axis_of_pair = [int(a) for a in axis_of_pair]
            n_axes = max(axis_of_pair, default=0) + 1
        else:
            axis_of_pair, n_axes = [0] * half, 1
        if len(axis_of_pair) != half or any(not 0 <= a < 4 for a in axis_of_pair) or n_axes > 4:
            raise ValueError("axis_of_pair must hold rot_dim / 2 = %d axes, each 0 .. 3" % half)
        self.rot_dim, self.n_axes = int(rot_dim), n_axes
        self._inv = (ctypes.c_double * max(half, 1))(*inv_freq)
        self._axis = (ctypes.c_uint8 * max(half, 1))(*axis_of_pair)
        self.c = HsaRopeParams(rot_dim=self.rot_dim, n_axes=n_axes, interleaved=int(bool(interleaved)),
                               scale=float(scale),
                               inv_freq=ctypes.cast(self._inv, ctypes.POINTER(ctypes.c_double)),
                               axis_of_pair=ctypes.cast(self._axis, ctypes.POINTER(ctypes.c_uint8)))
        self.ref = ctypes.byref(self.c)


# Small calls are bound by the host (a decode step's rotation is 3 us on the GPU), so the
# entry points below test everything a tensor has to be in one expression and go through
# the checks that name the fault only where that fails.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _good(t, dtype, shape):
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda \
        and t.is_contiguous()


def _expect(t, name, dtype, shape):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda
            and t.is_contiguous()):
        _need(t, name, dtype)
        _shape(t, name, shape)


def _err_ptr(t):
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.is_cuda and t.is_contiguous()
            and t.numel() >= 1):
        _need_err(t)
    return t.data_ptr()


def _need_rank(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor) or t.dim() != ndim:
        _need(t, name, dtype, ndim=ndim)


def _place(stream, *ts):
    """One device for all, the current one; -> its stream (an int or None)."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            _same_device(ts[0], *ts)
    if dev >= 0 and dev != _raw_device():
        raise ValueError("tensors on cuda:%d, but the current device is cuda:%d"
                         % (dev, torch.cuda.current_device()))
    if stream is None and dev >= 0 and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _head_rows(t, name, heads, d, n=None):
    """The token stride (elements) of a [n, heads, d] bf16 tensor whose tokens' heads are
    contiguous: dense, or a slice of wider rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != d or \
            (n is not None and shape[0] != n):
        raise ValueError("%s must have shape %s, got %s" % (
            name, ("n" if n is None else n, "heads" if heads is None else heads, d), tuple(shape)))
    s0, s1, s2 = t.stride()
    width = shape[1] * d
    if shape[0] <= 1:
        s0 = width
    if s2 != 1 or (s1 != d and shape[1] > 1) or s0 < width or s0 % 8:
        raise ValueError("%s: a token's heads must be contiguous and its stride a multiple of 8, "
                         "got strides %s" % (name, tuple(t.stride())))
    return s0


def _positions(rope, positions, n):
    if not _good(positions, torch.int32, (rope.n_axes, n)):
        _need(positions, "positions", torch.int32)
        if tuple(positions.shape) != (rope.n_axes, n) and not (
                rope.n_axes == 1 and tuple(positions.shape) == (n,)):
            raise ValueError("positions must have shape %s, got %s" % ((rope.n_axes, n),
                                                                       tuple(positions.shape)))


def hsa_rope(rope, q, k, positions, q_out=None, k_out=None, stream=None):
    """Turn the query heads q [n, Hq, d] and key heads k [n, Hkv, d] (bf16; dense, or slices
    of a QKV projection's rows) by positions [n_axes, n] int32 -> (q_out, k_out), dense.
    Either side may be None.  q_out may be a dense q itself (in place), and k_out k."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("give q, k or both")
    n, d = some.shape[0], some.shape[-1]
    Hq = Hkv = qs = ks = 0
    qp = kp = qo = ko = None
    if q is not None:
        qs, Hq = _head_rows(q, "q", None, d, n), q.shape[1]
        if q_out is None:
            q_out = _empty((n, Hq, d), q, stream)
        else:
            _expect(q_out, "q_out", torch.bfloat16, (n, Hq, d))
        qp, qo = q.data_ptr(), q_out.data_ptr()
    else:
        q_out = None
    if k is not None:
        ks, Hkv = _head_rows(k, "k", None, d, n), k.shape[1]
        if k_out is None:
            k_out = _empty((n, Hkv, d), k, stream)
        else:
            _expect(k_out, "k_out", torch.bfloat16, (n, Hkv, d))
        kp, ko = k.data_ptr(), k_out.data_ptr()
    else:
        k_out = None
    _positions(rope, positions, n)
    stream = _place(stream, positions, q, k, q_out, k_out)
    s = lib().hsa_rope(rope.ref, qp, qs, kp, ks, positions.data_ptr(), n, Hq, Hkv, d, qo, ko, stream)
    if s != HSA_OK:
        raise HsaError("hsa_rope", s)
    return q_out, k_out


def hsa_rope_kv_append(pool, layer, rope, q, k_new, v_new, cu_tokens, seq_idx, start_pos,
                       positions=None, q_out=None, k_out=None, dev_err=None, stream=None):
    """hsa_kv_append with the rotation on the way -> (q_out, k_out).  q [ntok, Hq, d] (or
    None: keys alone), k_new and v_new [ntok, Hkv, d] as in hsa_rope; positions [n_axes,
    ntok] int32, or None: each token's cache position on every axis.  k_out=False leaves
    the turned keys out (they go to the pool alone)."""
    Hq, Hkv, d = pool.Hq, pool.Hkv, pool.d
    ks = _head_rows(k_new, "k_new", Hkv, d)
    n = k_new.shape[0]
    vs = _head_rows(v_new, "v_new", Hkv, d, n)
    qs = 0
    qp = qo = ko = pos = None
    if q is not None:
        qs = _head_rows(q, "q", Hq, d, n)
        if q_out is None:
            q_out = _empty((n, Hq, d), q, stream)
        else:
            _expect(q_out, "q_out", torch.bfloat16, (n, Hq, d))
        qp, qo = q.data_ptr(), q_out.data_ptr()
    else:
        q_out = None
    if k_out is False:
        k_out = None
    else:
        if k_out is None:
            k_out = _empty((n, Hkv, d), k_new, stream)
        else:
            _expect(k_out, "k_out", torch.bfloat16, (n, Hkv, d))
        ko = k_out.data_ptr()
    if not isinstance(seq_idx, torch.Tensor) or seq_idx.dim() != 1:
        _need(seq_idx, "seq_idx", torch.int32, ndim=1)
    R = seq_idx.shape[0]
    _expect(seq_idx, "seq_idx", torch.int32, (R,))
    _expect(cu_tokens, "cu_tokens", torch.int32, (R + 1,))
    _expect(start_pos, "start_pos", torch.int32, (R,))
    if positions is not None:
        _positions(rope, positions, n)
        pos = positions.data_ptr()
    err = _err_ptr(dev_err)
    stream = _place(stream, k_new, q, v_new, cu_tokens, seq_idx, start_pos, positions, q_out, k_out,
                    dev_err, pool.block_tables)
    s = lib().hsa_rope_kv_append(pool.ref(), int(layer), rope.ref, qp, qs, k_new.data_ptr(), ks,
                                 v_new.data_ptr(), vs, pos, cu_tokens.data_ptr(),
                                 seq_idx.data_ptr(), start_pos.data_ptr(), R, n, qo, ko, err, stream)
    if s != HSA_OK:
        raise HsaError("hsa_rope_kv_append", s)
    return q_out, k_out


def hsa_decode_workspace_bytes(pool, B, T):
    return int(lib().hsa_decode_workspace_bytes(pool.ref(), int(B), int(T)))


def decode_workspace(pool, B, T, device="cuda"):
    """Zero-filled workspace for hsa_decode_attn (allocate once, reuse)."""
    n = hsa_decode_workspace_bytes(pool, B, T)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def _decode_shapes(pool, q, k_new, v_new, cached_len):
    B, T = q.shape[0], q.shape[1]
    _shape(q, "q", (B, T, pool.Hq, pool.d))
    _shape(k_new, "k_new", (B, T, pool.Hkv, pool.d))
    _shape(v_new, "v_new", (B, T, pool.Hkv, pool.d))
    _shape(cached_len, "cached_len", (B,))
    _same_device(q, k_new, v_new, cached_len)


def hsa_decode_attn(pool, layer, q, k_new, v_new, cached_len, scale, out=None, workspace=None,
                    max_ctas=0, dev_err=None, stream=None, append=False, early_pool_read=False):
    """Decode attention (hsa_decode_attn; with append=True hsa_decode_attn_append).
    early_pool_read=True calls hsa_decode_attn_ex with HSA_DECODE_EARLY_POOL_READ: the
    caller guarantees that the kernel queued just before on the stream does not write
    cached_len, ring_row or this layer's ring."""
    _need(q, "q", torch.bfloat16, ndim=4)
    _need(k_new, "k_new", torch.bfloat16, ndim=4)
    _need(v_new, "v_new", torch.bfloat16, ndim=4)
    _need(cached_len, "cached_len", torch.int32, ndim=1)
    B, T = q.shape[0], q.shape[1]
    _decode_shapes(pool, q, k_new, v_new, cached_len)
    if out is None:
        out = _empty(q.shape, q, stream)
    _need(out, "out", torch.bfloat16, ndim=4)
    _shape(out, "out", q.shape)
    if workspace is None:
        workspace = _made(lambda: decode_workspace(pool, B, T, device=q.device), q, stream)
    _need(workspace, "workspace", torch.uint8)
    _need_err(dev_err)
    _same_device(q, out, workspace, dev_err)
    args = (pool.ref(), int(layer), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(cached_len), B, T,
            float(scale), _ptr(out), _ptr(workspace), workspace.numel(), int(max_ctas))
    if early_pool_read:
        opts = HSA_DECODE_EARLY_POOL_READ | (HSA_DECODE_APPEND if append else 0)
        name = "hsa_decode_attn_ex"
        s = lib().hsa_decode_attn_ex(*args, opts, _ptr(dev_err), _stream(stream))
    else:
        name = "hsa_decode_attn_append" if append else "hsa_decode_attn"
        s = getattr(lib(), name)(*args, _ptr(dev_err), _stream(stream))
    _check(name, s)
    return out


def hsa_decode_attn_append(pool, layer, q, k_new, v_new, cached_len, scale, out=None,
                           workspace=None, max_ctas=0, dev_err=None, stream=None,
                           early_pool_read=False):
    """Decode attention, then the T new K/V rows of every sequence appended."""
    return hsa_decode_attn(pool, layer, q, k_new, v_new, cached_len, scale, out=out,
                           workspace=workspace, max_ctas=max_ctas, dev_err=dev_err,
                           stream=stream, append=True, early_pool_read=early_pool_read)


def hsa_decode_attn_noalloc(pool, layer, q, k_new, v_new, cached_len, scale, out, max_ctas=0,
                            dev_err=None, stream=None):
    """hsa_decode_attn with the library's own fixed device scratch: for callers that
    cannot allocate device memory where they run decode (no workspace argument).
    `out` must be supplied; the call itself allocates nothing.  The first call on a
    device should come before any stream capture; calls that could overlap on the
    GPU share one scratch array and must be serialised."""
    _need(q, "q", torch.bfloat16, ndim=4)
    _need(k_new, "k_new", torch.bfloat16, ndim=4)
    _need(v_new, "v_new", torch.bfloat16, ndim=4)
    _need(cached_len, "cached_len", torch.int32, ndim=1)
    _need(out, "out", torch.bfloat16, ndim=4)
    _decode_shapes(pool, q, k_new, v_new, cached_len)
    _shape(out, "out", q.shape)
    _need_err(dev_err)
    _same_device(q, out, dev_err)
    B, T = q.shape[0], q.shape[1]
    s = lib().hsa_decode_attn_noalloc(pool.ref(), int(layer), _ptr(q), _ptr(k_new), _ptr(v_new),
                                      _ptr(cached_len), B, T, float(scale), _ptr(out),
                                      int(max_ctas), _ptr(dev_err), _stream(stream))
    _check("hsa_decode_attn_noalloc", s)
    return out


def hsa_decode_shared_workspace_bytes(pool, B, T, n_groups):
    return int(lib().hsa_decode_shared_workspace_bytes(pool.ref(), int(B), int(T), int(n_groups)))


def decode_shared_workspace(pool, B, T, n_groups, device="cuda"):
    """Workspace for hsa_decode_attn_shared (allocate once, reuse; zero-filled)."""
    n = hsa_decode_shared_workspace_bytes(pool, B, T, n_groups)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def hsa_decode_attn_shared(pool, layer, q, k_new, v_new, cached_len, cu_group, shared_len, scale,
                           out=None, workspace=None, max_ctas=0, dev_err=None, stream=None,
                           append=False, early_pool_read=False):
    """Decode attention of a batch whose group g, sequences cu_group[g] .. cu_group[g + 1] - 1,
    shares the pages of its first shared_len[g] tokens (cu_group [n_groups + 1] and shared_len
    [n_groups], device int32): hsa_decode_attn's results, with a full layer's shared pages
    read once a group."""
    _need_rank(q, "q", torch.bfloat16, 4)
    _need_rank(shared_len, "shared_len", torch.int32, 1)
    B, T, n_groups = q.shape[0], q.shape[1], shared_len.shape[0]
    Hq, Hkv, d = pool.Hq, pool.Hkv, pool.d
    _expect(q, "q", torch.bfloat16, (B, T, Hq, d))
    _expect(k_new, "k_new", torch.bfloat16, (B, T, Hkv, d))
    _expect(v_new, "v_new", torch.bfloat16, (B, T, Hkv, d))
    _expect(cached_len, "cached_len", torch.int32, (B,))
    _expect(cu_group, "cu_group", torch.int32, (n_groups + 1,))
    _expect(shared_len, "shared_len", torch.int32, (n_groups,))
    if out is None:
        out = _empty(q.shape, q, stream)
    else:
        _expect(out, "out", torch.bfloat16, (B, T, Hq, d))
    if workspace is None:
        workspace = _made(lambda: decode_shared_workspace(pool, B, T, n_groups, device=q.device), q,
                          stream)
    else:
        _need(workspace, "workspace", torch.uint8)
    err = _err_ptr(dev_err)
    stream = _place(stream, q, k_new, v_new, cached_len, cu_group, shared_len, out, workspace,
                    dev_err, pool.block_tables)
    opts = (HSA_DECODE_APPEND if append else 0) | \
        (HSA_DECODE_EARLY_POOL_READ if early_pool_read else 0)
    s = lib().hsa_decode_attn_shared(pool.ref(), int(layer), q.data_ptr(), k_new.data_ptr(),
                                     v_new.data_ptr(), cached_len.data_ptr(), cu_group.data_ptr(),
                                     shared_len.data_ptr(), n_groups, B, T, float(scale),
                                     out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                     int(max_ctas), opts, err, stream)
    if s != HSA_OK:
        raise HsaError("hsa_decode_attn_shared", s)
    return out


def hsa_prefill_attn(pool, layer, q, k_new, v_new, cu_rows, prefix_len, seq_idx, max_chunk,
                     scale, out=None, dev_err=None, stream=None):
    _need(q, "q", torch.bfloat16, ndim=3)
    _need(k_new, "k_new", torch.bfloat16, ndim=3)
    _need(v_new, "v_new", torch.bfloat16, ndim=3)
    for n, t in (("cu_rows", cu_rows), ("prefix_len", prefix_len), ("seq_idx", seq_idx)):
        _need(t, n, torch.int32, ndim=1)
    R = seq_idx.shape[0]
    rows = q.shape[0]
    _shape(q, "q", (rows, pool.Hq, pool.d))
    _shape(k_new, "k_new", (rows, pool.Hkv, pool.d))
    _shape(v_new, "v_new", (rows, pool.Hkv, pool.d))
    _shape(cu_rows, "cu_rows", (R + 1,))
    _shape(prefix_len, "prefix_len", (R,))
    if out is None:
        out = _empty(q.shape, q, stream)
    _need(out, "out", torch.bfloat16, ndim=3)
    _shape(out, "out", q.shape)
    _need_err(dev_err)
    _same_device(q, k_new, v_new, cu_rows, prefix_len, seq_idx, out, dev_err)
    s = lib().hsa_prefill_attn(pool.ref(), int(layer), _ptr(q), _ptr(k_new), _ptr(v_new),
                               _ptr(cu_rows), _ptr(prefix_len), _ptr(seq_idx), R, q.shape[0],
                               int(max_chunk), float(scale), _ptr(out), _ptr(dev_err),
                               _stream(stream))
    _check("hsa_prefill_attn", s)
    return out


def _weight_rows(w, name, rows, heads):
    """w_stride of weights [rows, heads, w_stride] (fp32, w_stride a multiple of 4)."""
    _need_rank(w, name, torch.float32, 3)
    n = w.shape[2]
    _expect(w, name, torch.float32, (w.shape[0] if rows is None else rows,
                                     w.shape[1] if heads is None else heads, n))
    if n % 4:
        raise ValueError("%s: the row length must be a multiple of 4, got %d" % (name, n))
    return n


def hsa_decode_weights_workspace_bytes(pool, B, T, w_stride):
    return int(lib().hsa_decode_weights_workspace_bytes(pool.ref(), int(B), int(T), int(w_stride)))


def decode_weights_workspace(pool, B, T, w_stride, device="cuda"):
    """Workspace for hsa_decode_attn_weights (allocate once, reuse; any contents)."""
    n = hsa_decode_weights_workspace_bytes(pool, B, T, w_stride)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def hsa_decode_attn_weights(pool, layer, q, k_new, v_new, cached_len, scale, w, w_prev=None, decay=1.0,
                            out=None, workspace=None, max_ctas=0, dev_err=None, stream=None,
                            append=False):
    """Decode attention over a full layer that also weighs its keys: w [B, Hkv, w_stride] fp32
    becomes decay * w_prev + the softmax weight that the step's queries give each position
    (w_prev: the same shape, w itself, or None: nothing before).  -> out [B, T, Hq, d]."""
    _need_rank(q, "q", torch.bfloat16, 4)
    B, T = q.shape[0], q.shape[1]
    Hq, Hkv, d = pool.Hq, pool.Hkv, pool.d
    _expect(q, "q", torch.bfloat16, (B, T, Hq, d))
    _expect(k_new, "k_new", torch.bfloat16, (B, T, Hkv, d))
    _expect(v_new, "v_new", torch.bfloat16, (B, T, Hkv, d))
    _expect(cached_len, "cached_len", torch.int32, (B,))
    stride = _weight_rows(w, "w", B, Hkv)
    prev = None
    if w_prev is not None:
        _expect(w_prev, "w_prev", torch.float32, (B, Hkv, stride))
        prev = w_prev.data_ptr()
    if out is None:
        out = _empty(q.shape, q, stream)
    else:
        _expect(out, "out", torch.bfloat16, (B, T, Hq, d))
    if workspace is None:
        workspace = _made(lambda: decode_weights_workspace(pool, B, T, stride, device=q.device), q, stream)
    else:
        _need(workspace, "workspace", torch.uint8)
    err = _err_ptr(dev_err)
    stream = _place(stream, q, k_new, v_new, cached_len, w, w_prev, out, workspace, dev_err,
                    pool.block_tables)
    s = lib().hsa_decode_attn_weights(pool.ref(), int(layer), q.data_ptr(), k_new.data_ptr(),
                                      v_new.data_ptr(), cached_len.data_ptr(), B, T, float(scale),
                                      out.data_ptr(), prev, float(decay), w.data_ptr(), stride,
                                      workspace.data_ptr(), workspace.numel(), int(max_ctas),
                                      HSA_DECODE_APPEND if append else 0, err, stream)
    if s != HSA_OK:
        raise HsaError("hsa_decode_attn_weights", s)
    return out


def hsa_prefill_weights_workspace_bytes(pool, R, window):
    return int(lib().hsa_prefill_weights_workspace_bytes(pool.ref(), int(R), int(window)))


def prefill_weights_workspace(pool, R, window, device="cuda"):
    """Workspace for hsa_prefill_weights (allocate once, reuse; any contents)."""
    n = hsa_prefill_weights_workspace_bytes(pool, R, window)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def hsa_prefill_weights(pool, layer, q, cu_rows, kv_len, seq_idx, window, scale, w, w_prev=None,
                        decay=1.0, workspace=None, dev_err=None, stream=None):
    """After a chunk's append: w [batch, Hkv, w_stride] fp32, rows seq_idx, becomes decay * w_prev
    + the softmax weight that the last `window` queries of each request give every position of
    its sequence's kv_len[r] tokens.  q [rows, Hq, d], cu_rows [R + 1] as in hsa_prefill_attn
    -> w."""
    _need_rank(q, "q", torch.bfloat16, 3)
    _need_rank(seq_idx, "seq_idx", torch.int32, 1)
    R, rows = seq_idx.shape[0], q.shape[0]
    _expect(q, "q", torch.bfloat16, (rows, pool.Hq, pool.d))
    _expect(cu_rows, "cu_rows", torch.int32, (R + 1,))
    _expect(kv_len, "kv_len", torch.int32, (R,))
    _expect(seq_idx, "seq_idx", torch.int32, (R,))
    batch = pool.block_tables.shape[0]
    stride = _weight_rows(w, "w", batch, pool.Hkv)
    prev = None
    if w_prev is not None:
        _expect(w_prev, "w_prev", torch.float32, (batch, pool.Hkv, stride))
        prev = w_prev.data_ptr()
    if workspace is None:
        workspace = _made(lambda: prefill_weights_workspace(pool, R, window, device=q.device), q, stream)
    else:
        _need(workspace, "workspace", torch.uint8)
    err = _err_ptr(dev_err)
    stream = _place(stream, q, cu_rows, kv_len, seq_idx, w, w_prev, workspace, dev_err, pool.block_tables)
    s = lib().hsa_prefill_weights(pool.ref(), int(layer), q.data_ptr(), cu_rows.data_ptr(),
                                  kv_len.data_ptr(), seq_idx.data_ptr(), R, rows, int(window),
                                  float(scale), prev, float(decay), w.data_ptr(), stride,
                                  workspace.data_ptr(), workspace.numel(), err, stream)
    if s != HSA_OK:
        raise HsaError("hsa_prefill_weights", s)
    return w


def hsa_kv_select(w, kv_len, seq_idx, budget, sinks=0, recent=0, reach=0, keep=None, new_len=None,
                  dev_err=None, stream=None):
    """The positions of a budget that stay -> (keep [R, heads, budget] int32, ascending, -1
    past new_len; new_len [R] int32).  w [batch, heads, w_stride] fp32: request r is row
    seq_idx[r], of kv_len[r] positions.  The first `sinks` and the last `recent` always stay;
    the others by the largest weight among a position and `reach` neighbours on each side."""
    stride = _weight_rows(w, "w", None, None)
    _need_rank(seq_idx, "seq_idx", torch.int32, 1)
    R, heads, budget = seq_idx.shape[0], w.shape[1], int(budget)
    _expect(seq_idx, "seq_idx", torch.int32, (R,))
    _expect(kv_len, "kv_len", torch.int32, (R,))
    if budget < 0:
        raise ValueError("budget must not be negative")
    if keep is None:
        keep = _empty((R, heads, budget), seq_idx, stream)
    else:
        _expect(keep, "keep", torch.int32, (R, heads, budget))
    if new_len is None:
        new_len = _empty((R,), seq_idx, stream)
    else:
        _expect(new_len, "new_len", torch.int32, (R,))
    err = _err_ptr(dev_err)
    stream = _place(stream, w, kv_len, seq_idx, keep, new_len, dev_err)
    s = lib().hsa_kv_select(w.data_ptr(), stride, w.shape[0], heads, kv_len.data_ptr(),
                            seq_idx.data_ptr(), R, budget, int(sinks), int(recent), int(reach),
                            keep.data_ptr(), new_len.data_ptr(), err, stream)
    if s != HSA_OK:
        raise HsaError("hsa_kv_select", s)
    return keep, new_len


def hsa_kv_compact(pool, layer, keep, new_len, seq_idx, dst_tables, w=None, w_dst=None, dev_err=None,
                   stream=None):
    """Copy the K and V rows of a full layer at keep [R, Hkv or 1, budget] (positions of
    sequence seq_idx[r], the first new_len[r] of them) to positions 0, 1, ... of the pages
    dst_tables [R, dst_blocks] int32, and the weights w [batch, Hkv, w_stride] to w_dst."""
    _need_rank(keep, "keep", torch.int32, 3)
    _need_rank(dst_tables, "dst_tables", torch.int32, 2)
    R, heads, budget = keep.shape
    if heads != 1 and heads != pool.Hkv:
        raise ValueError("keep must have %d heads or one, got %d" % (pool.Hkv, heads))
    _expect(keep, "keep", torch.int32, (R, heads, budget))
    _expect(new_len, "new_len", torch.int32, (R,))
    _expect(seq_idx, "seq_idx", torch.int32, (R,))
    _expect(dst_tables, "dst_tables", torch.int32, (R, dst_tables.shape[1]))
    wp = wd = None
    stride = 0
    if (w is None) != (w_dst is None):
        raise ValueError("give w and w_dst, or neither")
    if w is not None:
        batch = pool.block_tables.shape[0]
        stride = _weight_rows(w, "w", batch, pool.Hkv)
        _expect(w_dst, "w_dst", torch.float32, (batch, pool.Hkv, stride))
        wp, wd = w.data_ptr(), w_dst.data_ptr()
    err = _err_ptr(dev_err)
    stream = _place(stream, keep, new_len, seq_idx, dst_tables, w, w_dst, dev_err, pool.block_tables)
    s = lib().hsa_kv_compact(pool.ref(), int(layer), keep.data_ptr(), heads, budget,
                             new_len.data_ptr(), seq_idx.data_ptr(), R, dst_tables.data_ptr(),
                             dst_tables.shape[1], wp, wd, stride, err, stream)
    if s != HSA_OK:
        raise HsaError("hsa_kv_compact", s)


def hsa_swa_prefetch(pool, layer, host_k, host_v, host_row, seq_idx, dev_err=None, stream=None):
    """Copy SWA ring rows of one sliding layer from pinned host memory into the
    device ring pool (row host_row[i] -> ring row of sequence seq_idx[i])."""
    for n, t in (("host_k", host_k), ("host_v", host_v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.is_cuda:
            raise TypeError("%s must be a bf16 host tensor" % n)
        if not t.is_pinned() or not t.is_contiguous():
            raise ValueError("%s must be pinned and contiguous" % n)
    if host_k.shape != host_v.shape or host_k.dim() != 4 or \
            tuple(host_k.shape[1:]) != (pool.Hkv, pool.W, pool.d):
        raise ValueError("host_k / host_v must be [n_host_rows, Hkv, W, d]")
    _need(host_row, "host_row", torch.int32, ndim=1)
    _need(seq_idx, "seq_idx", torch.int32, ndim=1)
    if host_row.shape != seq_idx.shape:
        raise ValueError("host_row and seq_idx must have the same length")
    _need_err(dev_err)
    _same_device(host_row, seq_idx, dev_err)
    s = lib().hsa_swa_prefetch(pool.ref(), int(layer), ctypes.c_void_p(host_k.data_ptr()),
                               ctypes.c_void_p(host_v.data_ptr()), host_k.shape[0],
                               _ptr(host_row), _ptr(seq_idx), host_row.shape[0], _ptr(dev_err),
                               _stream(stream))
    _check("hsa_swa_prefetch", s)


def hsa_window_safe_len(match_len, swa_slot_pos, W, out=None, stream=None):
    _need(match_len, "match_len", torch.int32, ndim=1)
    _need(swa_slot_pos, "swa_slot_pos", torch.int32, ndim=2)
    n = match_len.shape[0]
    if swa_slot_pos.shape != (n, W):
        raise ValueError("swa_slot_pos must be [n, W]")
    if out is None:
        out = _empty(match_len.shape, match_len, stream)
    _need(out, "out", torch.int32)
    _shape(out, "out", match_len.shape)
    _same_device(match_len, swa_slot_pos, out)
    s = lib().hsa_window_safe_len(_ptr(match_len), _ptr(swa_slot_pos), n, int(W), _ptr(out),
                                  _stream(stream))
    _check("hsa_window_safe_len", s)
    return out


def hsa_window_safe_len_bitmap(match_len, live_off, live, W, out=None, stream=None):
    _need(match_len, "match_len", torch.int32, ndim=1)
    _need(live_off, "live_off", torch.int64, ndim=1)
    _need(live, "live", torch.uint8, ndim=1)
    n = match_len.shape[0]
    if live_off.shape[0] != n + 1:
        raise ValueError("live_off must be [n+1]")
    if out is None:
        out = _empty(match_len.shape, match_len, stream)
    _need(out, "out", torch.int32)
    _shape(out, "out", match_len.shape)
    _same_device(match_len, live_off, live, out)
    s = lib().hsa_window_safe_len_bitmap(_ptr(match_len), _ptr(live_off), _ptr(live), n, int(W),
                                         _ptr(out), _stream(stream))
    _check("hsa_window_safe_len_bitmap", s)
    return out


def _i32_host(a, name):
    """A contiguous host int32 tensor of a one-dimensional sequence of ints (or a
    tensor).  Values outside the int32 range are refused, not wrapped."""
    t = a if isinstance(a, torch.Tensor) else torch.as_tensor(a)
    if t.is_cuda:
        raise ValueError("%s must be host memory" % name)
    if t.dim() > 1:
        raise ValueError("%s must be one-dimensional, got shape %s" % (name, tuple(t.shape)))
    if t.numel() == 0:
        return torch.zeros(0, dtype=torch.int32)
    if t.is_floating_point() or t.is_complex():
        raise ValueError("%s must hold integers, got %s" % (name, t.dtype))
    if t.dtype != torch.int32:
        lo, hi = int(t.min()), int(t.max())
        if lo < -2 ** 31 or hi > 2 ** 31 - 1:
            raise ValueError("%s holds values outside the int32 range" % name)
    return t.to(torch.int32).contiguous().view(-1)


class PrefixTree:
    """Host prefix tree of include/hsa_tree.h (Full index + SWA ring liveness).

    Methods mirror the C calls; token and slot arrays are host int32.
    ``window_safe(...)`` matches a batch on the host and computes every request's
    window-safe length on the GPU with hsa_window_safe_len.
    """

    def __init__(self, W, n_ring_rows):
        self.W = int(W)
        h = ctypes.c_void_p()
        _check("hsa_ptree_create", lib().hsa_ptree_create(self.W, int(n_ring_rows),
                                                           ctypes.byref(h)))
        self._h = h

    def close(self):
        if self._h is not None and self._h.value:
            lib().hsa_ptree_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def match(self, tokens, lock=False, take_ring=False):
        """-> (match_len, full_slots[match_len], ring_row, swa_slot_pos[W], lock_handle)."""
        tok = _i32_host(tokens, "tokens")
        n = tok.numel()
        slots = torch.empty(max(n, 1), dtype=torch.int32)
        pos = torch.empty(self.W, dtype=torch.int32)
        m, r, hnd = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
        _check("hsa_ptree_match", lib().hsa_ptree_match(
            self._h, ctypes.c_void_p(tok.data_ptr()), n, int(bool(lock)), int(bool(take_ring)),
            ctypes.byref(m), ctypes.c_void_p(slots.data_ptr()), ctypes.byref(r),
            ctypes.c_void_p(pos.data_ptr()), ctypes.byref(hnd)))
        return m.value, slots[:m.value].clone(), r.value, pos, hnd.value

    def match_batch(self, seqs):
        """-> (match_len [n], ring_row [n], swa_slot_pos [n, W]) host int32, read-only."""
        parts = [_i32_host(x, "tokens") for x in seqs]
        off = torch.zeros(len(seqs) + 1, dtype=torch.int64)
        if seqs:
            off[1:] = torch.cumsum(torch.tensor([t.numel() for t in parts], dtype=torch.int64), 0)
        flat = torch.cat(parts) if parts else torch.zeros(0, dtype=torch.int32)
        n = len(seqs)
        m = torch.empty(max(n, 1), dtype=torch.int32)
        r = torch.empty(max(n, 1), dtype=torch.int32)
        pos = torch.empty(max(n, 1), self.W, dtype=torch.int32)
        _check("hsa_ptree_match_batch", lib().hsa_ptree_match_batch(
            self._h, ctypes.c_void_p(flat.data_ptr()) if flat.numel() else None,
            ctypes.c_void_p(off.data_ptr()), n, ctypes.c_void_p(m.data_ptr()),
            ctypes.c_void_p(r.data_ptr()), ctypes.c_void_p(pos.data_ptr())))
        return m[:n], r[:n], pos[:n]

    def window_safe(self, seqs, device="cuda", stream=None):
        """Window-safe length of each request: host match, one GPU launch."""
        m, r, pos = self.match_batch(seqs)
        if m.numel() == 0:
            return m
        out = hsa_window_safe_len(m.to(device), pos.to(device), self.W, stream=stream)
        return out.cpu()

    def insert(self, tokens, full_slots, ring_row=-1, swa_slot_pos=None):
        """-> (dup_slots to free, ring_kept)."""
        tok = _i32_host(tokens, "tokens")
        sl = _i32_host(full_slots, "full_slots")
        if tok.numel() != sl.numel():
            raise ValueError("tokens and full_slots differ in length")
        n = tok.numel()
        pos = None
        if ring_row >= 0:
            pos = _i32_host(swa_slot_pos, "swa_slot_pos")
            if pos.numel() != self.W:
                raise ValueError("swa_slot_pos must hold W entries")
        dup = torch.empty(max(n, 1), dtype=torch.int32)
        nd, kept = ctypes.c_int32(), ctypes.c_int32()
        _check("hsa_ptree_insert", lib().hsa_ptree_insert(
            self._h, ctypes.c_void_p(tok.data_ptr()), ctypes.c_void_p(sl.data_ptr()), n,
            int(ring_row), None if pos is None else ctypes.c_void_p(pos.data_ptr()),
            ctypes.c_void_p(dup.data_ptr()), ctypes.byref(nd), ctypes.byref(kept)))
        return dup[:nd.value].clone(), bool(kept.value)

    def unlock(self, handle):
        _check("hsa_ptree_unlock", lib().hsa_ptree_unlock(self._h, int(handle)))

    def evict_full(self, n_tokens, slot_cap=None, row_cap=None):
        """-> (freed Full slots, freed ring rows).  The default capacities are what the
        tree holds, so every evictable leaf fits."""
        if slot_cap is None or row_cap is None:
            cached, rows, _ = self.stats()
            slot_cap = min(max(cached, 1), (1 << 31) - 1) if slot_cap is None else slot_cap
            row_cap = max(rows, 1) if row_cap is None else row_cap
        fs = torch.empty(max(slot_cap, 1), dtype=torch.int32)
        fr = torch.empty(max(row_cap, 1), dtype=torch.int32)
        ns, nr = ctypes.c_int32(), ctypes.c_int32()
        _check("hsa_ptree_evict_full", lib().hsa_ptree_evict_full(
            self._h, int(n_tokens), ctypes.c_void_p(fs.data_ptr()), int(slot_cap),
            ctypes.byref(ns), ctypes.c_void_p(fr.data_ptr()), int(row_cap), ctypes.byref(nr)))
        return fs[:ns.value].clone(), fr[:nr.value].clone()

    def evict_swa(self, n_rows):
        fr = torch.empty(max(int(n_rows), 1), dtype=torch.int32)
        nf = ctypes.c_int32()
        _check("hsa_ptree_evict_swa", lib().hsa_ptree_evict_swa(
            self._h, int(n_rows), ctypes.c_void_p(fr.data_ptr()), ctypes.byref(nf)))
        return fr[:nf.value].clone()

    def stats(self):
        """-> (cached tokens, ring rows held, nodes)."""
        c, rh, nn = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _check("hsa_ptree_stats", lib().hsa_ptree_stats(self._h, ctypes.byref(c),
                                                        ctypes.byref(rh), ctypes.byref(nn)))
        return c.value, rh.value, nn.value
