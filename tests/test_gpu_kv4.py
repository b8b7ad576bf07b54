"""GPU parity of the 4-bit key/value cache (ifq_kv4_append, ifq_kv4_read, ifq_kv4_attention) with the float64
oracle, its device-side range checks, and a decode step that runs the whole path."""
import math

import numpy as np
import pytest
import torch

import bit_complex_quantized_b200 as Q
import oracle as O
from oracle import fourbit as F
from ifq_testlib import DEV, gpu_quantize, run_gemv, status_word, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.load()


class Case:
    """A cache of sequences with given lengths and new tokens, on the device and as oracle codes.  fill: what the
    pages hold where no token was written."""

    def __init__(self, lens, news, heads, dim, page, seed=0, n_new=None, fill=0xFF, uniform=False, extra_cols=0):
        self.lens, self.news, self.heads, self.dim, self.page = lens, news, heads, dim, page
        rng = self.rng = np.random.default_rng(seed)
        B = len(lens)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages).astype(np.int32)
        table = np.full((B, max(1, max(need)) + extra_cols), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.records = np.full((pages, heads, page // 16, 32 * dim + 256), fill, np.uint8)
        offs = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.offs, self.used = offs, int(offs[-1])
        self.rows = max(1, self.used) + 2          # two rows that belong to no sequence
        self.n_new = max(1, max(news)) if n_new is None else n_new
        self.d_records = to_dev(self.records)
        self.d_table, self.d_lens, self.d_offs = to_dev(table), to_dev(np.array(lens, np.int32)), to_dev(offs)
        self.cache = Q.Kv4Cache(self.d_records, self.d_table, self.d_lens, dim, n_new=self.n_new, rows=self.rows,
                                new_offsets=None if uniform else self.d_offs)

    def planes(self, sharp=False):
        """Keys and values of the new tokens: k_re, k_im, v_re, v_im float32 [rows][heads dim]."""
        out = []
        for i in range(4):
            x = self.rng.standard_normal((self.rows, self.heads * self.dim)).astype(np.float32)
            if sharp and i < 2:
                x[:, ::7] *= 8
            out.append(x)
        return out

    def put(self, planes):
        """The oracle's append into self.records."""
        for b, (length, new) in enumerate(zip(self.lens, self.news)):
            for i in range(new):
                pos, row = length - new + i, self.offs[b] + i
                for h in range(self.heads):
                    cut = slice(h * self.dim, (h + 1) * self.dim)
                    k = F.kv4_quantize(np.stack([planes[0][row, cut], planes[1][row, cut]]))
                    v = F.kv4_quantize(np.stack([planes[2][row, cut], planes[3][row, cut]]))
                    rec = self.records[self.table[b, pos // self.page], h, (pos % self.page) // 16]
                    F.kv4_put(rec, pos % 16, k, v)

    def fill_random(self, spread=1.0):
        """Random contents of every page, written by the oracle's rules: codes and finite parameters."""
        r = self.rng
        self.records[:] = r.integers(0, 256, self.records.shape, dtype=np.uint8)
        par = self.records[..., 32 * self.dim:]
        s = F.bf16_bits(((r.random(par.shape[:-1] + (64,)) * 0.3 + 0.02) * spread).astype(np.float32))
        m = F.bf16_bits((-r.random(par.shape[:-1] + (64,)) * 3 * spread).astype(np.float32))
        par[:] = np.stack([s, m], axis=-1).reshape(par.shape[:-1] + (128,)).view(np.uint8)
        self.d_records.copy_(to_dev(self.records))

    def head(self, b, h):
        """(keys, values) codes of head h of sequence b, by address."""
        pages = self.table[b, :-(-self.lens[b] // self.page)]
        rec = self.records[pages, h].reshape(-1, 32 * self.dim + 256)
        k, v = F.kv4_get(rec, self.dim)
        return tuple(x[:self.lens[b]] for x in k), tuple(x[:self.lens[b]] for x in v)

    def attention(self, shared, scale=None, q=None, status=None, stream=None, q_scale=1.0):
        width = self.heads * shared * self.dim
        if q is None:
            q = [(q_scale * self.rng.standard_normal((self.rows, width))).astype(np.float32) for _ in range(2)]
        self.q, self.scale = q, 1 / math.sqrt(2 * self.dim) if scale is None else scale
        self.o = [torch.full((self.rows, width), 77.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        n = Q.ifq_kv4_attention_workspace_bytes(self.cache, self.heads * shared)
        self.ws = torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device=DEV)
        self.d_q = [to_dev(x) for x in q]
        Q.ifq_kv4_attention(self.cache, *self.d_q, *self.o, scale=self.scale, workspace=self.ws, dev_status=status,
                            stream=stream)

    def check(self, shared, skip=()):
        got = [x.float().cpu().numpy().astype(np.float64) for x in self.o]
        worst = 0.0
        for b, (length, new) in enumerate(zip(self.lens, self.news)):
            if b in skip or not new:
                continue
            rows = slice(self.offs[b], self.offs[b] + new)
            for h in range(self.heads):
                k, v = self.head(b, h)
                for a in range(h * shared, (h + 1) * shared):
                    cut = slice(a * self.dim, (a + 1) * self.dim)
                    q = np.concatenate([self.q[0][rows, cut], self.q[1][rows, cut]], axis=1).astype(np.float64)
                    o, bound = F.kv4_attention(q, k, v, length - new, self.scale)
                    have = np.concatenate([got[0][rows, cut], got[1][rows, cut]], axis=1)
                    # the output's own rounding to bf16: 2^-8 of the value
                    lim = bound + 2.0 ** -8 * (np.abs(o) + bound) + 1e-37
                    err = np.abs(have - o)
                    assert np.all(err <= lim), (b, h, a, float(np.max(err / lim)))
                    worst = max(worst, float(np.max(err / lim)))
        for x in got:
            assert np.all(x[self.used:] == 77.0), "rows behind the last sequence were written"
        return worst


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("lens,news,heads,page", [([1], [1], 1, 16), ([40, 17, 0, 3], [1, 1, 0, 3], 3, 16),
                                                  ([70, 33, 48], [50, 33, 2], 2, 48), ([130], [130], 5, 64)])
def test_append_and_read_bit_exact(lens, news, heads, page, dim):
    c = Case(lens, news, heads, dim, page, seed=dim + sum(lens), fill=0xA5)
    planes = c.planes(sharp=True)
    planes[0][0, :dim] = 0.25                       # a constant group: s = 0
    planes[2][0, :dim] = 0.0
    planes[1][0, :dim] = np.arange(dim) % 16 + 0.5  # m = 0.5, s = 1: exact steps
    if c.used > 1:
        t = (np.arange(dim) % 16).astype(np.float32) - np.float32(0.5)      # halves of steps of size 1
        t[:2] = 0, 15
        planes[3][1, :dim] = np.where(np.arange(dim) % 5 < 2, t, np.nextafter(t, np.float32(20)))
        planes[3][1, :2] = 0, 15
    st = status_word()
    Q.ifq_kv4_append(c.cache, *[to_dev(x) for x in planes], dev_status=st)
    out = [torch.full((c.rows, heads * dim), 55.0, device=DEV) for _ in range(4)]
    Q.ifq_kv4_read(c.cache, *out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.put(planes)
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)
    for x, o in zip(planes, out):
        n, s, m = F.kv4_quantize(x[:c.used].reshape(c.used, heads, dim))
        want = F.kv4_values(n, s, m).astype(np.float32).reshape(c.used, heads * dim)
        have = o.cpu().numpy()
        np.testing.assert_array_equal(have[:c.used], want)
        assert np.all(have[c.used:] == 55.0)


def test_append_range_and_nonfinite():
    c = Case([16], [16], 1, 64, 16, seed=5, fill=0)
    planes = c.planes()
    big = np.float32(3.4e38)
    planes[0][0, :3] = big, -big, 1.0               # rounds past the largest bf16: saturates
    planes[0][1, :2] = np.nan, np.inf
    planes[1][2] *= np.float32(1e-38)
    planes[1][3] *= np.float32(1e-42)
    planes[2][4] *= np.float32(1e30)
    planes[3][5, 1:] = planes[3][5, 1:] * np.float32(1e-6) + np.float32(1000.0)
    st = status_word()
    Q.ifq_kv4_append(c.cache, *[to_dev(x) for x in planes], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    c.put(planes)
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)


@pytest.mark.parametrize("new", [3, 16])
def test_append_widest_groups(new):
    """Groups whose spread passes float32: x - m overflows where the quotient does not."""
    c = Case([16], [new], 1, 64, 16, seed=7, fill=0)
    planes = c.planes()
    rng = np.random.default_rng(new)
    big = np.float32(3.38e38)
    for i, x in enumerate(planes):
        x[:new] = rng.uniform(-1, 1, (new, 64)).astype(np.float32) * big
        x[0, :2] = -big, big                               # steps of 2 big / 15: 0 is half way between two of them
        x[0, 2:8] = 0.0, 1e-45, -1e-45, 1e-30, -1e-30, 1.0
        x[1, :2] = 1e-45, big                              # one-sided: no overflow, the smallest minimum
        x[1, 2:] = np.abs(x[1, 2:])
    st = status_word()
    Q.ifq_kv4_append(c.cache, *[to_dev(x) for x in planes], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.put(planes)
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)


@pytest.mark.parametrize("B,heads,dim,page", [(64, 9, 32, 48), (90, 5, 64, 16), (128, 3, 32, 64), (50, 16, 128, 32)])
def test_append_many_heads_at_once(B, heads, dim, page):
    """Prompts large enough for several heads a block leave the records that appending 15 tokens at a time leaves."""
    rng = np.random.default_rng(B)
    news = [int(rng.integers(0, 200)) for _ in range(B - 1)] + [200]
    lens = [n + int(rng.integers(0, 40)) for n in news]
    c = Case(lens, news, heads, dim, page, seed=B, fill=0x5A)
    x = [torch.randn(c.rows, heads * dim, device=DEV) for _ in range(4)]
    x[0][3, 5], x[2][7, 1] = float("nan"), float("inf")
    st = status_word()
    Q.ifq_kv4_append(c.cache, *x, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    have = c.d_records.clone()
    c.d_records.copy_(to_dev(c.records))
    for done in range(0, 200, 15):
        part = [min(15, max(0, n - done)) for n in news]
        rows = torch.cat([torch.arange(c.offs[b] + done, c.offs[b] + done + n) for b, n in enumerate(part)]).to(DEV)
        if len(rows) == 0:
            break
        upto = np.array([length - new + min(new, done + 15) for length, new in zip(lens, news)], np.int32)
        offs = np.concatenate([[0], np.cumsum(part)]).astype(np.int32)
        cache = Q.Kv4Cache(c.d_records, c.d_table, to_dev(upto), dim, n_new=15, rows=len(rows), new_offsets=to_dev(offs))
        Q.ifq_kv4_append(cache, *[p[rows].contiguous() for p in x])
    torch.cuda.synchronize()
    assert torch.equal(have, c.d_records)


def test_append_takes_column_slices():
    """k and v as column slices of one wide output (a fused q, k, v product)."""
    c = Case([5, 9], [2, 1], 2, 64, 16, seed=6, fill=1)
    wide = [torch.randn(c.rows, 4 * 128, device=DEV) for _ in range(2)]
    cut = [wide[0][:, 128:256], wide[1][:, 128:256], wide[0][:, 256:384], wide[1][:, 256:384]]
    Q.ifq_kv4_append(c.cache, *cut)
    torch.cuda.synchronize()
    c.put([x.cpu().numpy() for x in cut])
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("lens,news,heads,shared,page", [
    ([1], [1], 1, 1, 16), ([15, 16, 17, 31, 32, 33], [1] * 6, 2, 1, 16), ([300, 0, 129, 1], [1, 0, 1, 1], 3, 8, 48),
    ([128, 127, 5], [4, 3, 5], 2, 3, 64), ([1000], [2], 1, 5, 256), ([40, 700], [16, 9], 1, 7, 32)])
def test_attention(lens, news, heads, shared, page, dim):
    c = Case(lens, news, heads, dim, page, seed=dim + len(lens))
    c.fill_random()
    st = status_word()
    c.attention(shared, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.check(shared)
    first = [x.clone() for x in c.o]
    c.attention(shared, q=c.q)
    torch.cuda.synchronize()
    for a, b in zip(first, c.o):
        assert torch.equal(a, b)


@pytest.mark.parametrize("q_scale", [1e-6, 6.0, 60.0])
def test_attention_flat_and_peaked(q_scale):
    c = Case([2000, 513], [1, 1], 2, 64, 64, seed=9)
    c.fill_random()
    c.attention(2, q_scale=q_scale)
    torch.cuda.synchronize()
    c.check(2)


def test_attention_long_and_split():
    """Many splits of long ragged sequences next to an empty one and a single token."""
    c = Case([20011, 1, 0, 4097], [1, 1, 0, 1], 1, 64, 64, seed=3, extra_cols=7)
    c.fill_random()
    assert Q.ifq_kv4_attention_workspace_bytes(c.cache, 8) > 0
    c.attention(8)
    torch.cuda.synchronize()
    c.check(8)


@pytest.mark.parametrize("B,shared,dim", [(128, 6, 64), (129, 1, 64), (200, 8, 32), (100, 5, 128)])
def test_attention_many_sequences(B, shared, dim):
    """More CTAs than the GPU holds: one long sequence (many records a warp, its page numbers fetched 32 at a time)
    among short and empty ones, wherever it stands in the batch."""
    lens, news = [1 + b % 3 for b in range(B)], [1] * B
    lens[B // 2], lens[3], news[3], lens[5] = 20003, 0, 0, 777
    c = Case(lens, news, 4, dim, 16 if B == 129 else 64, seed=B)
    c.fill_random()
    c.attention(shared)
    torch.cuda.synchronize()
    c.lens = lens
    first = [x.clone() for x in c.o]
    c.check(shared)
    c.attention(shared, q=c.q)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, c.o))


def test_attention_more_sequences_than_are_counted():
    """More sequences than the kernel counts by length: a CTA per head and tile of rows."""
    B = 1100
    lens, news = [1 + b % 5 for b in range(B)], [1] * B
    lens[700], lens[9], news[9] = 3000, 0, 0
    c = Case(lens, news, 1, 32, 16, seed=31)
    c.fill_random()
    c.attention(2)
    torch.cuda.synchronize()
    c.check(2)


def test_attention_replayed_while_lengths_grow():
    """A captured call over more splits than a cluster holds, replayed with longer sequences; a second cache's call
    runs at the same time on another stream with a workspace of its own."""
    c, other = Case([5000, 9], [1, 1], 1, 64, 64, seed=20, extra_cols=40), Case([3000], [1], 2, 64, 32, seed=21)
    c.fill_random()
    other.fill_random()
    spare = sorted(set(range(c.records.shape[0])) - set(c.table[c.table >= 0].tolist()))
    assert len(spare) == 2
    cols = (c.table[0] >= 0).sum()
    c.table[0, cols], c.d_table[0, cols] = spare[0], spare[0]
    c.attention(8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.ifq_kv4_attention(c.cache, *c.d_q, *c.o, scale=c.scale, workspace=c.ws)
    side = torch.cuda.Stream()
    for step in range(3):
        c.lens = [5000 + 7 * step, 9 + step]
        c.d_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        other.attention(3, stream=side, q=getattr(other, "q", None))
        torch.cuda.synchronize()
        c.check(8)
        other.check(3)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_attention_scales(scale):
    c = Case([70, 33], [1, 2], 2, 32, 16, seed=22)
    c.fill_random()
    c.attention(2, scale=scale)
    torch.cuda.synchronize()
    c.check(2)


@pytest.mark.parametrize("spread", [2.0 ** -60, 2.0 ** 60])
def test_attention_value_range(spread):
    """Stored values far from 1 (keys too: q is scaled against them)."""
    c = Case([300], [1], 2, 64, 16, seed=23)
    c.fill_random(spread)
    c.attention(2, q_scale=1.0 / spread)
    torch.cuda.synchronize()
    c.check(2)


def test_attention_huge_query_counts_as_not_finite():
    c = Case([100, 90], [1, 1], 1, 64, 16, seed=24)
    c.fill_random()
    q = [np.random.default_rng(i).standard_normal((c.rows, 64)).astype(np.float32) for i in range(2)]
    q[1][0, 3] = 3e38
    st = status_word()
    c.attention(1, q=q, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    assert torch.isnan(c.o[0][0]).all() and torch.isnan(c.o[1][0]).all()
    c.check(1, skip=(0,))


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attention_scale_not_finite(scale):
    c = Case([100], [2], 1, 64, 16, seed=25)
    c.fill_random()
    st = status_word()
    c.attention(1, scale=scale, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    for x in c.o:
        assert torch.isnan(x[:2]).all() and (x[2:] == 77.0).all()


@pytest.mark.parametrize("lens,news,heads,shared,dim", [
    ([9000, 5003, 37, 0], [16, 3, 0, 0], 2, 3, 64), ([20001], [5], 1, 8, 32), ([3000, 9001, 1], [1, 16, 1], 3, 5, 128),
    ([700] * 60 + [9000], [1] * 60 + [2], 8, 8, 64), ([1] * 30 + [12000] + [40] * 30, [1] * 61, 8, 1, 64)])
def test_attention_cut_pairs(lens, news, heads, shared, dim):
    """Runs that cut pairs, where sequences have fewer tiles of rows than the call allows for; fewer and more pairs than
    blocks."""
    c = Case(lens, news, heads, dim, 64, seed=len(lens) + dim, n_new=16 if len(lens) < 5 else None)
    c.fill_random()
    assert Q.ifq_kv4_attention_workspace_bytes(c.cache, heads * shared) > 0
    c.attention(shared)
    torch.cuda.synchronize()
    c.check(shared)
    first = [x.clone() for x in c.o]
    c.attention(shared, q=c.q)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, c.o))


@pytest.mark.parametrize("B", [1024, 1025])
def test_attention_most_sequences_that_are_counted(B):
    """The most sequences whose runs are counted, and one more: a block per pair whatever the lengths."""
    lens, news = [1 + b % 4 for b in range(B)], [1] * B
    lens[B - 1], lens[100], lens[1], news[1] = 3001, 999, 0, 0
    c = Case(lens, news, 2, 32, 16, seed=B)
    c.fill_random()
    st = status_word()
    c.attention(2, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.check(2)


@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 24])
def test_attention_value_outlier(ratio):
    """A key with values `ratio` times larger than all others and a weight of almost nothing."""
    c = Case([70], [1], 1, 64, 16, seed=26)
    c.fill_random()
    at = c.table[0, 1], 0, 0                     # token 16
    par = c.records[at][32 * 64:].view(np.uint16).reshape(2, 16, 4)
    par[1, 0] = F.bf16_bits(F.bf16_value(par[1, 0]) * np.float32(ratio))
    par[0, 0, 1::2] = F.bf16_bits(np.full(2, -1e4, np.float32))     # its key: far below the others
    c.d_records.copy_(to_dev(c.records))
    q = [np.abs(c.rng.standard_normal((c.rows, 64))).astype(np.float32) for _ in range(2)]
    c.attention(1, q=q)
    torch.cuda.synchronize()
    c.check(1)


def test_attention_ignores_what_lies_behind():
    """NaN parameters and codes behind the last token, in its own record and in others, never reach an output."""
    c = Case([33, 7], [1, 2], 2, 64, 32, seed=4, fill=0xFF)
    planes = c.planes()
    c.lens, keep = list(c.news), c.lens
    # write all tokens of both sequences through the library, in two calls
    for start, upto in ((0, 20), (20, 33)):
        lens = [min(n, upto) for n in keep]
        news = [max(0, n - start) if n > start else 0 for n in lens]
        cc = Case(lens, news, 2, 64, 32, seed=4, n_new=64)
        cc.table = c.table
        cache = Q.Kv4Cache(c.d_records, c.d_table, to_dev(np.array(lens, np.int32)), 64, n_new=64, rows=cc.rows,
                           new_offsets=cc.d_offs)
        p = cc.planes()
        Q.ifq_kv4_append(cache, *[to_dev(x) for x in p])
        cc.records = c.records
        cc.put(p)
    c.lens = keep
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)
    c.attention(4)
    torch.cuda.synchronize()
    c.check(4)
    assert planes is not None


def test_attention_bad_numbers_in_device_memory():
    """Offsets, lengths and pages outside their ranges are skipped and reported; other sequences stay right."""
    c = Case([50, 40, 30, 20, 10], [1, 1, 2, 1, 1], 2, 64, 16, seed=8)
    c.fill_random()
    lens, table = c.d_lens.clone(), c.d_table.clone()
    lens[0] = 10 ** 6                                # longer than the table
    lens[1] = 0                                      # shorter than its new tokens
    table[3, 0] = 10 ** 6                            # a page that does not exist: its keys are left out
    cache = Q.Kv4Cache(c.d_records, table, lens, 64, n_new=2, rows=c.rows, new_offsets=c.d_offs)
    good, c.cache = c.cache, cache
    st = status_word()
    c.attention(2, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_RANGE
    c.check(2, skip=(0, 1, 3))
    for x in c.o:
        assert torch.all(x[c.offs[0]:c.offs[2]] == 0)
    # sequence 3 sees positions 16..19 only
    got = torch.cat([x[c.offs[3], :64].float() for x in c.o]).cpu().numpy()
    k, v = c.head(3, 0)
    q = np.concatenate([x[c.offs[3], :64] for x in c.q])[None].astype(np.float64)
    o, bound = F.kv4_attention(q, tuple(x[16:] for x in k), tuple(x[16:] for x in v), 3, c.scale)
    assert np.all(np.abs(got - o[0]) <= bound[0] + 2.0 ** -8 * (np.abs(o[0]) + bound[0]))
    # appending: nothing outside the good sequences' tokens is written
    before = c.d_records.clone()
    st.zero_()
    planes = c.planes()
    Q.ifq_kv4_append(cache, *[to_dev(x) for x in planes], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_RANGE
    save = c.news
    c.news = [0, 0, 2, 1, 1]                          # sequence 3's new token lies in its second, good page
    c.put(planes)
    c.news = save
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)
    assert not torch.equal(before, c.d_records)
    # offsets: decreasing, past the rows, more than n_new
    for bad in ([0, 1, 2, 4, 3, 5], [0, 1, 2, 4, 5, 10 ** 6], [0, 3, 3, 4, 5, 6], [-1, 1, 2, 4, 5, 6]):
        offs = to_dev(np.array(bad, np.int32))
        c.cache = Q.Kv4Cache(c.d_records, c.d_table, c.d_lens, 64, n_new=2, rows=c.rows, new_offsets=offs)
        st.zero_()
        c.attention(2, status=st)
        torch.cuda.synchronize()
        assert int(st) & Q.IFQ_DEV_RANGE
    c.cache = good
    st.zero_()
    c.attention(2, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.check(2)


def test_bad_numbers_among_many_sequences():
    """The same checks where the work is counted over the batch: bad lengths, offsets and pages change nothing for
    the others, and every bad kind is reported."""
    B, heads, shared = 160, 4, 8
    rng = np.random.default_rng(40)
    lens = [int(n) for n in rng.integers(1, 400, B)]
    news = [int(min(n, 1 + i % 3)) for i, n in enumerate(lens)]
    c = Case(lens, news, heads, 64, 32, seed=40, n_new=3)
    c.fill_random()
    bad_len, empty, bad_page = 17, 60, 101
    d_lens, table = c.d_lens.clone(), c.d_table.clone()
    d_lens[bad_len] = 10 ** 7
    d_lens[empty] = -5
    table[bad_page] = c.records.shape[0]
    c.cache = Q.Kv4Cache(c.d_records, table, d_lens, 64, n_new=3, rows=c.rows, new_offsets=c.d_offs)
    st = status_word()
    c.attention(shared, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_RANGE
    c.check(shared, skip=(bad_len, empty, bad_page))
    for b in (bad_len, empty, bad_page):
        for x in c.o:
            assert torch.all(x[c.offs[b]:c.offs[b + 1]] == 0)
    offs = c.d_offs.clone()
    offs[50], offs[90] = c.rows + 7, -3              # two sequences each lose their rows
    c.cache = Q.Kv4Cache(c.d_records, c.d_table, c.d_lens, 64, n_new=3, rows=c.rows, new_offsets=offs)
    st.zero_()
    c.attention(shared, q=c.q, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_RANGE
    c.check(shared, skip=(49, 50, 89, 90))
    for b in (49, 50, 89, 90):                       # never written
        for x in c.o:
            assert torch.all(x[c.offs[b]:c.offs[b + 1]] == 77.0)


def test_attention_nonfinite_query_stays_in_its_row():
    c = Case([100, 90], [1, 1], 1, 64, 16, seed=11)
    c.fill_random()
    q = [np.random.default_rng(i).standard_normal((c.rows, 3 * 64)).astype(np.float32) for i in range(2)]
    q[0][0, 64 + 5] = np.nan                          # sequence 0, head 1
    st = status_word()
    c.attention(3, q=q, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    assert torch.isnan(c.o[0][0, 64:128]).all() and torch.isnan(c.o[1][0, 64:128]).all()
    for x in c.o:
        assert torch.isfinite(x[0, :64]).all() and torch.isfinite(x[0, 128:]).all()
    c.check(3, skip=(0,))


def test_offsets_past_32_bits():
    """Pages more than 4 GB into the cache."""
    dim, heads, page = 64, 8, 64
    pages = (5 << 30) // (heads * (page // 16) * 2304)
    rec = torch.zeros(Q.Kv4Cache.records_shape(pages, heads, page, dim), dtype=torch.uint8, device=DEV)
    assert rec.numel() > 1 << 32
    c = Case([100], [100], heads, dim, page, seed=1)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    planes = c.planes()
    cache = Q.Kv4Cache(rec, table, c.d_lens, dim, n_new=100, rows=c.rows)
    Q.ifq_kv4_append(cache, *[to_dev(x) for x in planes])
    c.put(planes)
    got = rec[pages - 2:].flip(0).cpu().numpy()
    want = c.records[c.table[0]]
    np.testing.assert_array_equal(got[0], want[0])
    D = 2 * dim                                      # the second page holds 36 tokens: compare what they stand for
    for h in range(heads):
        for a, b in zip(F.kv4_get(got[1, h], dim), F.kv4_get(want[1, h], dim)):
            for x, y in zip(a, b):
                np.testing.assert_array_equal(x[:36], y[:36])
    assert not rec[:pages - 2].any() and D == 128
    step = Case([100], [1], heads, dim, page, seed=1)
    step.records, step.table = c.records, c.table
    step.cache = Q.Kv4Cache(rec, table, step.d_lens, dim, n_new=1, rows=step.rows)
    step.attention(2)
    torch.cuda.synchronize()
    step.check(2)


# ------------------------------------------------------------------ the path as it is used
def test_decode_steps_through_the_library():
    """Three decode steps of two sequences: q, k, v by the 2-bit products with their rotation, append,
    attention, and an output layer in 4 bits, captured once as a graph and replayed while the lengths grow.
    Every call's result is checked against float64 from the buffers that the call read."""
    rng = np.random.default_rng(12)
    heads, shared, dim, B, hidden = 2, 2, 64, 2, 128
    n_q, n_kv = heads * shared * dim, heads * dim

    def weights(N, K):
        return [(0.05 * rng.standard_normal((N, K))).astype(np.float32) for _ in range(2)]

    x = [torch.zeros(B, hidden, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    layers, mats = [], []
    for N in (n_q, n_kv, n_kv):
        u, w = weights(N, hidden), weights(N, hidden)
        (cu, su), (cw, sw) = gpu_quantize([tuple(map(to_dev, u)), tuple(map(to_dev, w))], 2)
        theta = rng.random((B, N)).astype(np.float32) * 6
        d = dict(codes_u=cu, scales_u=su, codes_w=cw, scales_w=sw, N=N, K=hidden, x_re=x[0], x_im=x[1],
                 y_re=torch.empty(B, N, device=DEV), y_im=torch.empty(B, N, device=DEV),
                 rot_re=to_dev(np.cos(theta)), rot_im=to_dev(np.sin(theta)))
        layers.append(d)
        mats.append((O.dequantize(cu.cpu().numpy(), su.cpu().numpy()), O.dequantize(cw.cpu().numpy(), sw.cpu().numpy()),
                     np.cos(theta).astype(np.float64) + 1j * np.sin(theta)))
    R = (0.02 * rng.standard_normal((2 * hidden, 2 * n_q))).astype(np.float32)
    cs, ss = Q.w4_shapes(*R.shape, 64)
    codes, scales = torch.empty(cs, dtype=torch.uint8, device=DEV), torch.empty(ss, dtype=torch.bfloat16, device=DEV)
    Q.ifq_w4_quantize([(to_dev(R), codes, scales)], 64)
    o = [torch.empty(B, n_q, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = dict(codes=codes, scales=scales, rows=2 * hidden, cols=2 * n_q, x_re=o[0], x_im=o[1],
               y_re=torch.empty(B, hidden, device=DEV), y_im=torch.empty(B, hidden, device=DEV))
    c = Case([4, 20], [1, 1], heads, dim, 16, seed=2, uniform=True, extra_cols=1)
    c.fill_random()
    c.d_table[0, 1], c.table[0, 1] = c.records.shape[0] - 1, c.records.shape[0] - 1
    free = sorted(set(range(c.records.shape[0])) - set(c.table[c.table >= 0].tolist()))
    if c.table[0, 1] in c.table[1]:
        c.d_table[0, 1] = c.table[0, 1] = free[0]
    cache = Q.Kv4Cache(c.d_records, c.d_table, c.d_lens, dim)
    ws = torch.empty(max(16, Q.ifq_kv4_attention_workspace_bytes(cache, heads * shared)), dtype=torch.uint8, device=DEV)
    gws = torch.zeros(max(16, Q.ifq_gemv_workspace_bytes(layers, 2, B)), dtype=torch.uint8, device=DEV)
    st = status_word()

    def step():
        Q.ifq_gemv(layers, 2, B, workspace=gws, dev_status=st)
        q, k, v = layers
        Q.ifq_kv4_append(cache, k["y_re"], k["y_im"], v["y_re"], v["y_im"], dev_status=st)
        Q.ifq_kv4_attention(cache, q["y_re"], q["y_im"], *o, scale=0.09, workspace=ws, dev_status=st)
        Q.ifq_w4_gemv([out], 64, B, dev_status=st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        for t in x:
            t.copy_(torch.randn(B, hidden, device=DEV))
        graph.replay()
        c.d_lens += 1
        torch.cuda.synchronize()
        c.lens = [4 + n, 20 + n]
        xv = x[0].double().cpu().numpy() + 1j * x[1].double().cpu().numpy()
        for d, (U, W, rot) in zip(layers, mats):
            want = (xv @ U.T + xv.conj() @ W.T) * rot
            got = d["y_re"].double().cpu().numpy() + 1j * d["y_im"].double().cpu().numpy()
            absx = np.abs(xv.real) + np.abs(xv.imag)
            lim = 1e-5 * ((np.abs(U.real) + np.abs(U.imag) + np.abs(W.real) + np.abs(W.imag)).max() * absx.sum(1))
            assert np.all(np.abs(got - want) <= lim[:, None])
        planes = [layers[i][p].cpu().numpy() for i in (1, 2) for p in ("y_re", "y_im")]
        c.offs = np.array([0, 1, 2])
        c.put(planes)
        np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)
        c.q, c.scale, c.o, c.used = [layers[0][p].cpu().numpy() for p in ("y_re", "y_im")], 0.09, o, B
        c.check(shared)
        q4, s4 = F.w4_quantize(R, 64)
        Wv = F.w4_values(q4, s4, 64)
        ov = torch.cat(o, dim=1).double().cpu().numpy()
        y = torch.cat([out["y_re"], out["y_im"]], dim=1).double().cpu().numpy()
        assert np.all(np.abs(y - ov @ Wv.T) <= 32 * 2.0 ** -22 * (np.abs(ov) @ np.abs(Wv).T))
    assert int(st) == 0


# ------------------------------------------------------------------ what a call does not name
@pytest.mark.parametrize("n_new", [1, 8, 16, 32])
def test_idle_sequence_names_no_page(n_new):
    """A sequence without new tokens whose length ends inside a record of a page that was given back (-1): nothing of
    the call names that page, so no form of it reports a range, and the other sequence's tokens are written."""
    c = Case([37, 5 + n_new, 16], [0, n_new, 0], 3, 64, 16, seed=50 + n_new)
    c.fill_random()
    c.table[0, 2] = -1                               # the page of tokens 32..36
    c.d_table.copy_(to_dev(c.table))
    planes = c.planes()
    st = status_word()
    Q.ifq_kv4_append(c.cache, *[to_dev(x) for x in planes], dev_status=st)
    out = [torch.full((c.rows, 3 * 64), 55.0, device=DEV) for _ in range(4)]
    Q.ifq_kv4_read(c.cache, *out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.put(planes)
    np.testing.assert_array_equal(c.d_records.cpu().numpy(), c.records)
    for x, o in zip(planes, out):
        n, s, m = F.kv4_quantize(x[:c.used].reshape(c.used, 3, 64))
        np.testing.assert_array_equal(o.cpu().numpy()[:c.used], F.kv4_values(n, s, m).astype(np.float32).reshape(c.used, -1))
        assert torch.all(o[c.used:] == 55.0)
    if n_new <= Q.IFQ_KV4_MAX_NEW:
        c.attention(2, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        c.check(2, skip=(0,))


# ------------------------------------------------------------------ limits as documented
@pytest.mark.parametrize("scale", [1.0, 0.0625, -2.0])
def test_attention_query_limit(scale):
    """|scale q| of 2^99 is taken, the next float above it counts as not finite (the powers of two of the scale are
    exact, so nothing is rounded on the way there but the factor log2 e, which keeps the order)."""
    c = Case([40, 40, 40], [1, 1, 1], 1, 64, 16, seed=60)
    c.fill_random(spread=2.0 ** -90)                 # keys near 2^-90: scores of order 2^9
    q = [np.zeros((c.rows, 64), np.float32) for _ in range(2)]
    top = np.float32(2.0 ** 99 / abs(scale))
    q[0][0, 3], q[1][1, 7], q[1][2, 7] = top, np.nextafter(top, np.float32(np.inf)), -1.3 * top
    st = status_word()
    c.attention(1, q=q, scale=scale, status=st)
    torch.cuda.synchronize()
    assert int(st) == Q.IFQ_DEV_NONFINITE
    for x in c.o:
        assert torch.isfinite(x[0]).all() and torch.isnan(x[1:3]).all()
    q[1][1:3] = 0
    st.zero_()
    c.attention(1, q=q, scale=scale, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c.check(1, skip=(0,))
    assert all(torch.isfinite(x[0]).all() for x in c.o)


# ------------------------------------------------------------------ two calls at once
def test_attention_of_two_caches_at_once():
    """Two caches' calls on two streams, one of them a captured graph, with a workspace each and nothing on the host
    between them: each has the result that it has alone, over and over."""
    a, b = Case([20011, 9, 4097], [1, 1, 1], 2, 64, 64, seed=70), Case([9000, 12001], [2, 1], 3, 64, 32, seed=71)
    for c, shared in ((a, 8), (b, 3)):
        c.fill_random()
        c.attention(shared)
        torch.cuda.synchronize()
        c.check(shared)
        c.alone = [x.clone() for x in c.o]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        for _ in range(4):
            Q.ifq_kv4_attention(a.cache, *a.d_q, *a.o, scale=a.scale, workspace=a.ws)
    for _ in range(5):
        for c in (a, b):
            c.ws.fill_(0xFF)
            for x in c.o:
                x.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        for _ in range(4):
            Q.ifq_kv4_attention(b.cache, *b.d_q, *b.o, scale=b.scale, workspace=b.ws, stream=side)
        torch.cuda.synchronize()
        for c in (a, b):
            assert all(torch.equal(x, y) for x, y in zip(c.alone, c.o))


@pytest.mark.parametrize("scale,ok", [(2.0 ** 127, True), (-2.0 ** 127, True), (1.25 * 2.0 ** 127, False), (-3e38, False)])
def test_attention_largest_scale(scale, ok):
    """|scale| of 2^127 is taken, more counts as not finite (scale log2 e may pass float32)."""
    c = Case([50], [2], 1, 64, 16, seed=61)
    c.fill_random()
    st = status_word()
    c.attention(1, scale=scale, q_scale=2.0 ** -126, status=st)
    torch.cuda.synchronize()
    assert int(st) == (0 if ok else Q.IFQ_DEV_NONFINITE)
    if ok:
        c.check(1)
    else:
        assert all(torch.isnan(x[:2]).all() for x in c.o)


@pytest.mark.parametrize("shared,power", [(1, -110), (1, -121), (8, -121), (2, -124)])
def test_attention_smallest_values(shared, power):
    """Values whose scales lie near the end of float32's range keep the stated bound (no slack but bf16's own: half a
    step of its subnormal numbers is 2^-134)."""
    c = Case([300, 40], [1, 1], 2, 64, 16, seed=62)
    c.fill_random()
    par = c.records[..., 32 * 64 + 128:]
    bits = np.ascontiguousarray(par).view(np.uint16)
    par[:] = F.bf16_bits(F.bf16_value(bits) * np.float32(2.0 ** power)).view(np.uint8)
    c.d_records.copy_(to_dev(c.records))
    c.attention(shared)
    torch.cuda.synchronize()
    got = torch.stack(c.o).double().cpu().numpy()
    for b, length in enumerate(c.lens):
        for h in range(2):
            k, v = c.head(b, h)
            for a in range(h * shared, (h + 1) * shared):
                cut = slice(a * 64, (a + 1) * 64)
                q = np.concatenate([x[b, cut] for x in c.q])[None].astype(np.float64)
                o, bound = F.kv4_attention(q, k, v, length - 1, c.scale)
                lim = bound[0] + 2.0 ** -8 * (np.abs(o[0]) + bound[0]) + 2.0 ** -134
                assert np.all(np.abs(np.concatenate(got[:, b, cut]) - o[0]) <= lim), (b, a)
