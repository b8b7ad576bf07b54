"""GPU parity of the 4-bit layers (ifq_w4_quantize, ifq_w4_dequantize, ifq_w4_gemv) with the float64 oracle."""
import numpy as np
import pytest
import torch

import bit_complex_quantized_b200 as Q
from oracle import fourbit as F
from ifq_testlib import DEV, status_word, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.load()


def quantize(Rs, group, status=None):
    """Device (codes, scales) of numpy or device layers; buffers start filled with another pattern."""
    items = []
    for R in Rs:
        R = to_dev(R) if isinstance(R, np.ndarray) else R
        cs, ss = Q.w4_shapes(*R.shape, group)
        items.append((R, torch.full(cs, 0xA5, dtype=torch.uint8, device=DEV),
                      torch.full(ss, -1, dtype=torch.int16, device=DEV)))
    Q.ifq_w4_quantize(items, group, dev_status=status)
    return [(c, s) for _, c, s in items]


def hard_weights(rows, cols, group, seed):
    """Normal weights with rows that are hard to quantize: exact halves of a step, neighbours of halves, zeros,
    subnormals, one large entry, the largest float32."""
    rng = np.random.default_rng(seed)
    R = (0.02 * rng.standard_normal((rows, cols))).astype(np.float32)
    half = np.tile(np.arange(group) % 14 - 6.5, cols // group).astype(np.float32)
    special = [half * np.float32(2.0 ** -9), None, np.zeros(cols, np.float32),
               R[0] * np.float32(1e-38), R[0] * np.float32(1e-42), None, None]
    step = np.float32(1.3671875)                   # a bf16 value: the halves of its steps, and their neighbours
    t = half * step
    special[1] = np.where(rng.integers(0, 2, cols) == 0, t, np.nextafter(t, np.float32(np.inf) * np.sign(t)))
    special[1] = np.where(rng.integers(0, 3, cols) == 0, np.nextafter(t, np.float32(0)), special[1])
    special[1].reshape(-1, group)[:, 0] = 7 * step
    special[0].reshape(-1, group)[:, 0] = 7 * np.float32(2.0 ** -9)
    special[5] = R[0].copy()
    special[5][::group] = 3.0e3
    special[6] = np.full(cols, np.finfo(np.float32).max, np.float32) * np.where(np.arange(cols) % 3 == 0, 1, -0.3)
    for i, s in enumerate(special):
        if i < rows:
            R[rows - 1 - i] = s
    return R


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shapes", [[(1, 128)], [(16, 128)], [(37, 256), (5, 1152)], [(250, 640)]])
def test_quantize_and_dequantize_bit_exact(shapes, group):
    Rs = [hard_weights(r, c, group, 10 * r + c) for r, c in shapes]
    got = quantize(Rs, group)
    outs = [torch.full(R.shape, -1, dtype=torch.int16, device=DEV) for R in Rs]
    Q.ifq_w4_dequantize([(c, s, o) for (c, s), o in zip(got, outs)], group)
    torch.cuda.synchronize()
    for R, (c, s), o in zip(Rs, got, outs):
        q, sb = F.w4_quantize(R, group)
        wc, ws = F.w4_pack(q, sb)
        np.testing.assert_array_equal(c.cpu().numpy(), wc)
        np.testing.assert_array_equal(s.cpu().numpy().view(np.uint16), ws)
        want = F.bf16_bits((np.repeat(F.bf16_value(sb), group, axis=1) * q.astype(np.float32)))
        # a zero code is +0 or -0 by the code's sign only where q = 0: compare values, then bits where nonzero
        have = o.cpu().numpy().view(np.uint16)
        np.testing.assert_array_equal(have & 0x7FFF, want & 0x7FFF)
        np.testing.assert_array_equal(have[q != 0], want[q != 0])


def test_quantize_nonfinite():
    R = hard_weights(20, 128, 64, 3)
    R[3, 5], R[4, 70], R[0] = np.nan, -np.inf, np.inf
    st = status_word()
    (c, s), = quantize([R], 64, st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    wc, ws = F.w4_pack(*F.w4_quantize(R, 64))
    np.testing.assert_array_equal(c.cpu().numpy(), wc)
    np.testing.assert_array_equal(s.cpu().numpy().view(np.uint16), ws)
    st.zero_()
    quantize([hard_weights(20, 128, 64, 3)], 64, st)
    torch.cuda.synchronize()
    assert int(st) == 0


def make_layer(rows, cols, group, B, planar_x, planar_y, rng, x=None):
    R = (0.02 * rng.standard_normal((rows, cols))).astype(np.float32)
    (codes, scales), = quantize([R], group)
    if x is None:
        x = rng.standard_normal((B, cols)).astype(np.float32)
    xt = torch.from_numpy(x).to(torch.bfloat16)
    d = dict(codes=codes, scales=scales, rows=rows, cols=cols, x_im=None, y_im=None)
    if planar_x:
        d["x_re"], d["x_im"] = xt[:, :cols // 2].contiguous().to(DEV), xt[:, cols // 2:].contiguous().to(DEV)
    else:
        d["x_re"] = xt.to(DEV)
    if planar_y:
        d["y_re"] = torch.full((B, rows // 2), 7e7, device=DEV)
        d["y_im"] = torch.full((B, rows // 2), 7e7, device=DEV)
    else:
        d["y_re"] = torch.full((B, rows), 7e7, device=DEV)
    q, s = F.w4_quantize(R, group)
    return d, F.w4_values(q, s, group), xt.float().numpy().astype(np.float64)


def check_layer(d, W, x, group):
    y = d["y_re"] if d["y_im"] is None else torch.cat([d["y_re"], d["y_im"]], dim=1)
    # exact products; at most one float32 rounding (2^-22 of the terms so far, truncation included) per matrix
    # instruction of a group, per group and per joined part, each of at most the sum of magnitudes
    steps = group / 16 + d["cols"] / group + 16
    bound = steps * 2.0 ** -22 * (np.abs(x) @ np.abs(W).T)
    err = np.abs(y.cpu().numpy().astype(np.float64) - x @ W.T)
    assert np.all(err <= bound + 1e-300), float(np.max(err / (bound + 1e-300)))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols,B,planar", [(2, 128, 1, True), (1, 128, 16, False), (130, 256, 3, True),
                                                (127, 384, 9, False), (512, 512, 8, True), (66, 4224, 16, True),
                                                (1000, 1408, 2, True), (257, 11008, 1, False), (48, 28672, 16, True)])
def test_gemv(rows, cols, group, B, planar):
    rng = np.random.default_rng(rows + cols + B)
    d, W, x = make_layer(rows, cols, group, B, planar, planar, rng)
    st = status_word()
    Q.ifq_w4_gemv([d], group, B, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    check_layer(d, W, x, group)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("count", [1, 9])
@pytest.mark.parametrize("B", [2, 3, 4, 5, 8, 9])
def test_gemv_batches(B, count, group):
    """The last and first batches of each form of the kernel, which differ in the rows of a CTA and in who fetches x;
    rows around a CTA's 64 and 128."""
    rng = np.random.default_rng(100 * B + count)
    made = [make_layer(r, 128 * (3 + i % 3), group, B, False, r % 2 == 0, rng)
            for i, r in enumerate([65, 64, 128, 129, 127, 63, 192, 193, 16][:count])]
    st = status_word()
    Q.ifq_w4_gemv([m[0] for m in made], group, B, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for m in made:
        check_layer(*m, group)


@pytest.mark.parametrize("B", [1, 7, 16])
def test_gemv_grouped_layers_and_mixed_planes(B):
    """Layers of one call with different shapes and plane forms; cols 64 (mod 128) splits the planes inside a tile."""
    rng = np.random.default_rng(B)
    group = 64
    made = [make_layer(r, c, group, B, px, py, rng) for r, c, px, py in
            [(4096, 1024, True, True), (2, 64, True, False), (301, 192, False, False), (48, 2816, False, True),
             (16, 320, True, True)]]
    Q.ifq_w4_gemv([m[0] for m in made], group, B)
    torch.cuda.synchronize()
    for d, W, x in made:
        check_layer(d, W, x, group)
    again = [m[0]["y_re"].clone() for m in made]
    many = [dict(m[0], y_re=torch.empty_like(m[0]["y_re"])) for m in made]
    Q.ifq_w4_gemv(many, group, B)
    torch.cuda.synchronize()
    for a, d in zip(again, many):
        assert torch.equal(a, d["y_re"])


def test_gemv_thirty_two_layers():
    rng = np.random.default_rng(0)
    made = [make_layer(2 * i + 2, 128, 128, 4, True, True, rng) for i in range(32)]
    Q.ifq_w4_gemv([m[0] for m in made], 128, 4)
    torch.cuda.synchronize()
    for d, W, x in made:
        check_layer(d, W, x, 128)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 100])
def test_gemv_activation_range(scale):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((3, 256)) * scale).astype(np.float32)
    d, W, xv = make_layer(40, 256, 32, 3, True, True, rng, x=x)
    Q.ifq_w4_gemv([d], 32, 3)
    torch.cuda.synchronize()
    check_layer(d, W, xv, 32)


def test_gemv_nonfinite_token_stays_in_its_row():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 256)).astype(np.float32)
    x[2, 7] = np.inf
    d, W, xv = make_layer(70, 256, 64, 5, True, False, rng, x=x)
    st = status_word()
    Q.ifq_w4_gemv([d], 64, 5, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    assert not torch.isfinite(d["y_re"][2]).any()
    keep = [0, 1, 3, 4]
    d["y_re"] = d["y_re"][keep]
    check_layer(d, W, xv[keep], 64)


def test_gemv_block_graph_and_stream():
    """The seven layers of a 7B-shaped block: one call, the same call on another stream, and captured and replayed
    on new activations, all give the same bits as separate calls."""
    rng = np.random.default_rng(4)
    group, B = 128, 1
    shapes = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]
    made = [make_layer(r, c, group, B, True, True, rng) for r, c in shapes]
    layers = [m[0] for m in made]
    Q.ifq_w4_gemv(layers, group, B)
    torch.cuda.synchronize()
    for d, W, x in made:
        check_layer(d, W, x, group)
    want = [torch.cat([d["y_re"], d["y_im"]]) for d in layers]
    side = torch.cuda.Stream()
    for d in layers:
        d["y_re"].zero_()
    side.wait_stream(torch.cuda.current_stream())
    Q.ifq_w4_gemv(layers, group, B, stream=side)
    side.synchronize()
    for d, w in zip(layers, want):
        assert torch.equal(torch.cat([d["y_re"], d["y_im"]]), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.ifq_w4_gemv(layers, group, B)
    for d in layers:
        d["x_re"].copy_(torch.randn_like(d["x_re"], dtype=torch.float32))
    graph.replay()
    torch.cuda.synchronize()
    for d, W, x in made:
        xv = torch.cat([d["x_re"], d["x_im"]], dim=1).float().cpu().numpy().astype(np.float64)
        check_layer(d, W, xv, group)


def test_gemv_two_calls_at_once():
    """Two calls on two streams share nothing: both give what they give alone."""
    rng = np.random.default_rng(8)
    a, Wa, xa = make_layer(2048, 2048, 128, 2, True, True, rng)
    b, Wb, xb = make_layer(1500, 4096, 128, 11, False, False, rng)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        Q.ifq_w4_gemv([a], 128, 2)
        Q.ifq_w4_gemv([b], 128, 11, stream=side)
    torch.cuda.synchronize()
    check_layer(a, Wa, xa, 128)
    check_layer(b, Wb, xb, 128)


def test_gemv_layer_set_repeats_the_call():
    rng = np.random.default_rng(9)
    made = [make_layer(r, 512, 64, 3, True, True, rng) for r in (64, 200, 1024)]
    layers = Q.W4LayerSet([m[0] for m in made], 64, 3)
    for _ in range(2):
        for d, _, _ in made:
            d["y_re"].fill_(-1.0)
        Q.ifq_w4_gemv(layers, 64, 3)
        torch.cuda.synchronize()
        for d, W, x in made:
            check_layer(d, W, x, 64)
    with pytest.raises(ValueError):
        Q.ifq_w4_gemv(layers, 64, 2)
