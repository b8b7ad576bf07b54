"""Host-side checks of the 4-bit layers and cache (no GPU needed): argument errors come back as status codes or
ValueError before any CUDA call, and the oracle's layout and quantizer hold their definitions."""
import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_complex_quantized_b200 as Q
from bit_complex_quantized_b200 import _lib as L
from oracle import fourbit as F

FAKE = 0x10000  # non-null, 16-byte aligned, never dereferenced by validation
OK, NULL, SHAPE, ALIGN, BATCH, WORKSPACE, COUNT = 0, 1, 2, 3, 5, 6, 9


def _tensor(**kw):
    d = dict(R=FAKE, rows=64, cols=128, codes=FAKE, scales=FAKE)
    d.update(kw)
    return L.W4Tensor(*[d[n] for n, _ in L.W4Tensor._fields_])


def _layer(**kw):
    d = dict(codes=FAKE, scales=FAKE, rows=64, cols=128, x_re=FAKE, x_im=FAKE, y_re=FAKE, y_im=FAKE)
    d.update(kw)
    return L.W4Layer(*[d[n] for n, _ in L.W4Layer._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(rows=0), SHAPE), (dict(cols=0), SHAPE),
    (dict(cols=96), SHAPE), (dict(cols=130), SHAPE), (dict(rows=(1 << 30) + 1), SHAPE),
    (dict(rows=1 << 30, cols=1 << 12), SHAPE), (dict(codes=FAKE + 8), ALIGN), (dict(scales=FAKE + 2), ALIGN)])
def test_w4_argument_errors(kw, status):
    lib = Q.load()
    assert lib.ifq_w4_quantize((L.W4Tensor * 1)(_tensor(**kw)), 1, 64, None, None) == status
    assert lib.ifq_w4_gemv((L.W4Layer * 1)(_layer(**kw)), 1, 64, 1, None, None) == status
    d = dict(codes=FAKE, scales=FAKE, rows=64, cols=128, w=FAKE)
    d.update(kw)
    assert lib.ifq_w4_dequantize((L.W4DqTensor * 1)(L.W4DqTensor(*[d[n] for n, _ in L.W4DqTensor._fields_])), 1, 64,
                                 None) == status


def test_w4_call_errors():
    lib = Q.load()
    one, lay = (L.W4Tensor * 1)(_tensor()), (L.W4Layer * 1)(_layer())
    assert lib.ifq_w4_quantize(None, 1, 64, None, None) == NULL
    assert lib.ifq_w4_quantize(one, 0, 64, None, None) == COUNT
    assert lib.ifq_w4_quantize(one, 33, 64, None, None) == COUNT
    for group in (0, 16, 48, 256):
        assert lib.ifq_w4_quantize(one, 1, group, None, None) == SHAPE
        assert lib.ifq_w4_gemv(lay, 1, group, 1, None, None) == SHAPE
    assert lib.ifq_w4_quantize((L.W4Tensor * 1)(_tensor(cols=192)), 1, 128, None, None) == SHAPE
    assert lib.ifq_w4_quantize((L.W4Tensor * 1)(_tensor(R=None)), 1, 64, None, None) == NULL
    assert lib.ifq_w4_quantize((L.W4Tensor * 1)(_tensor(R=FAKE + 4)), 1, 64, None, None) == ALIGN
    assert lib.ifq_w4_gemv(lay, 1, 64, 0, None, None) == BATCH
    assert lib.ifq_w4_gemv(lay, 1, 64, 17, None, None) == BATCH
    assert lib.ifq_w4_gemv((L.W4Layer * 1)(_layer(rows=63)), 1, 64, 1, None, None) == SHAPE   # planar y, odd rows
    for kw, status in ((dict(x_re=None), NULL), (dict(y_re=None), NULL), (dict(x_im=FAKE + 2), ALIGN),
                       (dict(y_im=FAKE + 4), ALIGN)):
        assert lib.ifq_w4_gemv((L.W4Layer * 1)(_layer(**kw)), 1, 64, 1, None, None) == status


def _cache(**kw):
    d = dict(records=FAKE, pages=10, page_tokens=64, kv_heads=4, dim=64, B=3, n_new=1, rows=3, page_table=FAKE,
             table_cols=8, kv_lens=FAKE, new_offsets=None)
    d.update(kw)
    return L.Kv4CacheDesc(*[d[n] for n, _ in L.Kv4CacheDesc._fields_])


def _append(c, ptrs=(FAKE,) * 4, ld=256):
    return Q.load().ifq_kv4_append(c if c is None else ctypes.byref(c), *ptrs, ld, None, None)


def _attend(c, heads=8, q=FAKE, o=FAKE, ldq=512, ldo=512, ws=FAKE, nb=1 << 40):
    return Q.load().ifq_kv4_attention(c if c is None else ctypes.byref(c), heads, q, q, ldq, 0.1, o, o, ldo, ws, nb, None,
                                      None)


@pytest.mark.parametrize("kw,status", [
    (dict(records=None), NULL), (dict(page_table=None), NULL), (dict(kv_lens=None), NULL), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(page_tokens=8), SHAPE), (dict(page_tokens=24), SHAPE),
    (dict(page_tokens=1 << 17), SHAPE), (dict(kv_heads=0), SHAPE), (dict(dim=48), SHAPE), (dict(dim=256), SHAPE),
    (dict(B=0), SHAPE), (dict(B=65536, rows=65536), SHAPE), (dict(n_new=0), BATCH), (dict(n_new=2), SHAPE), (dict(rows=2), SHAPE),
    (dict(rows=0), SHAPE), (dict(table_cols=0), SHAPE), (dict(table_cols=1 << 26, page_tokens=65536), SHAPE),
    (dict(records=FAKE + 8), ALIGN), (dict(kv_lens=FAKE + 2), ALIGN), (dict(new_offsets=FAKE + 1), ALIGN)])
def test_cache_argument_errors(kw, status):
    assert _append(_cache(**kw)) == status
    assert Q.load().ifq_kv4_read(ctypes.byref(_cache(**kw)), FAKE, FAKE, FAKE, FAKE, 256, None, None) == status
    assert _attend(_cache(**kw)) == status
    assert Q.load().ifq_kv4_attention_workspace_bytes(ctypes.byref(_cache(**kw)), 8) == 0


def test_cache_call_errors():
    lib, c = Q.load(), _cache()
    assert _append(None) == NULL and _attend(None) == NULL
    for i in range(4):
        ptrs = [FAKE] * 4
        ptrs[i] = None
        assert _append(c, ptrs) == NULL
        ptrs[i] = FAKE + 4
        assert _append(c, ptrs) == ALIGN
    assert _append(c, ld=255) == SHAPE and _append(c, ld=252) == SHAPE and _append(c, ld=258) == SHAPE
    assert _attend(c, heads=0) == SHAPE and _attend(c, heads=2) == SHAPE and _attend(c, heads=9) == SHAPE
    assert _attend(c, heads=4100) == SHAPE
    assert _attend(_cache(n_new=17, rows=51)) == BATCH
    assert _append(_cache(n_new=Q.IFQ_KV4_MAX_APPEND + 1, new_offsets=FAKE)) == BATCH
    assert _attend(c, q=None) == NULL and _attend(c, o=None) == NULL
    assert _attend(c, q=FAKE + 4) == ALIGN and _attend(c, o=FAKE + 2) == ALIGN
    assert _attend(c, ldq=508) == SHAPE and _attend(c, ldq=514) == SHAPE and _attend(c, ldo=513) == SHAPE
    need = lib.ifq_kv4_attention_workspace_bytes(ctypes.byref(_cache(table_cols=4096)), 8)
    assert need > 0
    assert _attend(_cache(table_cols=4096), nb=need - 1) == WORKSPACE
    assert _attend(_cache(table_cols=4096), ws=None) == WORKSPACE
    assert _attend(_cache(table_cols=4096), ws=FAKE + 8) == ALIGN


def test_python_refuses_wrong_tensors():
    R = torch.zeros(16, 128)
    cs, ss = Q.w4_shapes(16, 128, 64)
    codes, scales = torch.zeros(cs, dtype=torch.uint8), torch.zeros(ss, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        Q.ifq_w4_quantize([(R, codes, scales)], 64)                     # not on a GPU
    with pytest.raises(ValueError):
        Q.ifq_w4_quantize([(R, codes[:, :1], scales)], 64)
    with pytest.raises(ValueError):
        Q.ifq_w4_quantize([(R.double(), codes, scales)], 64)
    with pytest.raises(ValueError):
        Q.ifq_w4_quantize([(R[:, ::2], codes, scales)], 64)
    with pytest.raises(ValueError):
        Q.ifq_w4_quantize([(R, codes, scales)], 48)
    for call in (Q.ifq_w4_quantize, Q.ifq_w4_dequantize):
        with pytest.raises(Q.IfqError):
            call([], 64)
    with pytest.raises(Q.IfqError):
        Q.ifq_w4_gemv([], 64, 1)
    with pytest.raises(ValueError):
        Q.Kv4Cache(torch.zeros(2, 1, 1, 100, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32),
                   torch.zeros(1, dtype=torch.int32), 64)
    for n_new in (0, -1, 1 << 32 | 1):
        with pytest.raises(Q.IfqError):
            Q.Kv4Cache(torch.zeros(2, 1, 1, 32 * 64 + 256, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32), 64, n_new=n_new)


# ------------------------------------------------------------------ the oracle against the definitions
@pytest.mark.parametrize("rows,cols,group", [(16, 64, 32), (21, 192, 64), (33, 256, 128)])
def test_w4_layout_holds_every_entry_once(rows, cols, group):
    rng = np.random.default_rng(rows)
    q = rng.integers(-7, 8, (rows, cols)).astype(np.int8)
    s = rng.integers(0, 1 << 15, (rows, cols // group)).astype(np.uint16)
    codes, scales = F.w4_pack(q, s)
    assert (codes.shape, scales.shape) == Q.w4_shapes(rows, cols, group)
    seen = np.zeros(codes.size * 2, int)
    for r in range((rows + 15) // 16 * 16):
        for k in range(cols):
            at, bit = F.w4_code_place(r, k, cols)
            seen[2 * at + bit // 4] += 1
            assert (int(codes.flat[at]) >> bit & 15) - 8 == (q[r, k] if r < rows else 0)
    assert (seen == 1).all()


def test_kv4_layout_holds_every_entry_once():
    for dim in (32, 64, 128):
        D = 2 * dim
        seen = np.zeros(2 * 16 * D, int)
        for r in range(16):
            for d in range(D):
                for at, bit in (F.kv4_key_place(r, d), F.kv4_value_place(r, d, D)):
                    seen[2 * at + bit // 4] += 1
        assert (seen == 1).all()
        rng = np.random.default_rng(dim)
        rec = rng.integers(0, 256, 32 * dim + 256, dtype=np.uint8)
        x = rng.standard_normal((2, 2, dim)).astype(np.float32)
        k, v = F.kv4_quantize(x[0]), F.kv4_quantize(x[1])
        before = F.kv4_get(rec[None].copy(), dim)
        F.kv4_put(rec, 9, k, v)
        after = F.kv4_get(rec[None], dim)
        for a, b, new in zip(before, after, (k, v)):
            for x0, x1, y in zip(a, b, new):
                np.testing.assert_array_equal(x1[9], y)
                np.testing.assert_array_equal(np.delete(x0, 9, 0), np.delete(x1, 9, 0))


def _half_even(f):
    n = f.numerator // f.denominator
    rest = f - n
    return n + (rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2 == 1))


def test_quantizers_round_exact_quotients():
    """Codes against rational arithmetic, at halves of a step and their neighbours too."""
    rng = np.random.default_rng(0)
    R = rng.standard_normal((4, 64)).astype(np.float32)
    step = np.float32(0.3671875)
    R[1] = (np.arange(64) % 14 - np.float32(6.5)) * step
    R[2] = np.nextafter(R[1], np.float32(0))
    R[3] = np.nextafter(R[1], np.float32(9))
    R[1:, 0] = 7 * step
    q, s = F.w4_quantize(R, 32)
    for r in range(4):
        for k in range(64):
            sv = Fraction(float(F.bf16_value(s[r:r + 1, k // 32])[0]))
            assert q[r, k] == max(-7, min(7, _half_even(Fraction(float(R[r, k])) / sv)))
    x = rng.standard_normal((3, 64)).astype(np.float32)
    x[1] = np.arange(64) % 16 - np.float32(0.5)
    x[1, :2] = 0, 15
    x[2] = np.nextafter(x[1], np.float32(99))
    x[2, :2] = 0, 15
    n, s, m = F.kv4_quantize(x)
    for r in range(3):
        sv, mv = (Fraction(float(F.bf16_value(t[r:r + 1])[0])) for t in (s, m))
        for k in range(64):
            assert n[r, k] == max(0, min(15, _half_even((Fraction(float(x[r, k])) - mv) / sv)))


# ------------------------------------------------------------------ kernels that are launched while the one before ends
def test_kernels_that_follow_read_behind_their_wait():
    """A kernel that starts before the one in front of it has ended reads nothing through the read-only path, whose
    lines may be older than its wait, nor by loads that the compiler may move in front of the wait."""
    csrc = os.path.dirname(L.__file__) + "/csrc/"
    found = 0
    for name in sorted(os.listdir(csrc)):
        text = open(csrc + name).read()
        if "follow();" in text or name == "kv4_common.cuh":
            found += 1
            for load in ("__ldg(", "__ldcg(", "__ldca(", "ldg_stream(", "ld.global.nc"):
                assert load not in text, (name, load)
            assert "__ldcs(" not in text or "behind_wait(" in text
    assert found == 4                                 # w4_gemv, kv4_cache, kv4_attention and what the last two share


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("kw", [dict(pages=1 << 30, kv_heads=4), dict(pages=1 << 20, kv_heads=1024, page_tokens=65536),
                                dict(pages=(1 << 32) // 16, page_tokens=64, kv_heads=4)])
def test_cache_of_more_records_than_are_counted(kw):
    """Attention numbers records in 32 bits, and the last number is none."""
    c = _cache(**kw)
    width = c.kv_heads * 64
    assert c.pages * c.kv_heads * (c.page_tokens // 16) >= 1 << 32
    assert _append(c, ld=width) == SHAPE and _attend(c, heads=c.kv_heads, ldq=width, ldo=width) == SHAPE
    assert Q.load().ifq_kv4_attention_workspace_bytes(ctypes.byref(c), c.kv_heads) == 0
    # one page fewer is taken (a missing workspace is refused after the sizes: nothing is launched)
    c.pages = ((1 << 32) - 1) // (c.kv_heads * (c.page_tokens // 16))
    c.table_cols = (1 << 20) // c.page_tokens
    assert Q.load().ifq_kv4_attention_workspace_bytes(ctypes.byref(c), c.kv_heads) > 0
    assert _attend(c, heads=c.kv_heads, ldq=width, ldo=width, nb=0) == WORKSPACE
