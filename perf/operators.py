"""Cases of the 4-bit operators: layers with 4-bit weights and group scales (quantize, decode product) and a
key/value cache held in 4 bits (append, attention).

Each case runs either in a plain form (elementary torch operations in float32) or, with own = True, through
the entry points of bit_complex_quantized_b200.  The buffers are those of include/ifq.h in both.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16_MAX = 3.3895313892515355e38
# (byte, low/high nibble) of a 32-bit word of eight codes -> the code's position; and its inverse
WORD_ORDER = [0, 2, 4, 6, 1, 3, 5, 7]
WORD_PLACE = [0, 4, 1, 5, 2, 6, 3, 7]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one fake-quantization pass over the weights of a 7B-shaped attention layer (real 4096 x 4096)
        {"name": "w4_quantize_4096", "op": "w4_quantize", "rows": 4096, "cols": 4096, "group": 128},
        # a ragged row count (a vocabulary slice) at the finest group, the 7B-shaped FFN width
        {"name": "w4_quantize_ragged", "op": "w4_quantize", "rows": 10007, "cols": 11008, "group": 32},
        # the smallest decode call: one 256 x 256 complex layer's real form, one token; latency only
        {"name": "w4_gemv_small", "op": "w4_gemv", "shapes": "512x512", "group": 64, "B": 1, "planar": True},
        # one token through a 7B-shaped block kept in 4 bits: q, k, v, o, gate, up, down in one call
        {"name": "w4_gemv_block7b", "op": "w4_gemv",
         "shapes": "4096x4096 4096x4096 4096x4096 4096x4096 11008x4096 11008x4096 4096x11008",
         "group": 128, "B": 1, "planar": True},
        # a logits head over the concatenated planes for five requests: odd vocabulary, fine groups, plain rows
        {"name": "w4_gemv_head", "op": "w4_gemv", "shapes": "50021x4096", "group": 32, "B": 5, "planar": False},
        # sixteen requests through the 70B-shaped gate and down layers
        {"name": "w4_gemv_ffn70b_b16", "op": "w4_gemv", "shapes": "28672x8192 8192x28672", "group": 64, "B": 16,
         "planar": True},
        # one decode step of 16 requests, 8 key/value heads of 64 complex entries
        {"name": "kv4_append_step", "op": "kv4_append", "B": 16, "n_new": 1, "kv_heads": 8, "dim": 64, "page": 64,
         "max_len": 4096, "ragged": True},
        # prompts entering the cache: four requests of up to 2048 tokens, 32 heads (7B-shaped)
        {"name": "kv4_append_prompt", "op": "kv4_append", "B": 4, "n_new": 2048, "kv_heads": 32, "dim": 64, "page": 64,
         "max_len": 2500, "ragged": True},
        # one request early in its answer, 32 heads without sharing; latency counts
        {"name": "kv4_attn_short", "op": "kv4_attention", "B": 1, "n_new": 1, "kv_heads": 32, "shared": 1, "dim": 64,
         "page": 64, "max_len": 777, "ragged": False},
        # one request with a long context, 64 query heads on 8 key/value heads (70B-shaped)
        {"name": "kv4_attn_long", "op": "kv4_attention", "B": 1, "n_new": 1, "kv_heads": 8, "shared": 8, "dim": 64,
         "page": 256, "max_len": 131072, "ragged": False},
        # a serving batch of ragged lengths (an empty slot and a first token among them), 70B-shaped heads
        {"name": "kv4_attn_batch", "op": "kv4_attention", "B": 32, "n_new": 1, "kv_heads": 8, "shared": 8, "dim": 64,
         "page": 64, "max_len": 20000, "ragged": True},
        # checking four drafted tokens per request, small heads, pages that end inside a block of keys
        {"name": "kv4_attn_draft", "op": "kv4_attention", "B": 9, "n_new": 4, "kv_heads": 5, "shared": 3, "dim": 32,
         "page": 16, "max_len": 3001, "ragged": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w4_quantize", "w4_gemv", "w4_gemv", "kv4_append", "kv4_attention", "kv4_attention"])
    if op == "w4_quantize":
        group = rng.choice([32, 64, 128])
        unit = max(group, 64)
        return {"op": op, "rows": _log_int(rng, 1, 11008), "cols": unit * _log_int(rng, 1, 8192 // unit),
                "group": group}
    if op == "w4_gemv":
        group = rng.choice([32, 64, 128])
        planar = rng.random() < 0.6
        shapes = []
        for _ in range(rng.choice([1, 1, 2, 3, 7])):
            cols = 128 * _log_int(rng, 1, 86)
            rows = _log_int(rng, 2, 11008)
            shapes.append("%dx%d" % (rows + (rows & 1 if planar else 0), cols))
        return {"op": op, "shapes": " ".join(shapes), "group": group, "B": rng.randint(1, 16), "planar": planar}
    dim = rng.choice([32, 64, 64, 128])
    case = {"op": op, "B": _log_int(rng, 1, 32), "n_new": 1, "kv_heads": rng.choice([1, 2, 5, 8, 16, 32]), "dim": dim,
            "page": rng.choice([16, 32, 48, 64, 128, 256]), "max_len": 0, "ragged": rng.random() < 0.7}
    if op == "kv4_append":
        case["n_new"] = _log_int(rng, 1, 1024) if rng.random() < 0.6 else 1
        case["B"] = min(case["B"], max(1, 8192 * 64 * 32 // (case["n_new"] * case["kv_heads"] * dim)))
        case["max_len"] = case["n_new"] + _log_int(rng, 1, 4096)
        return case
    case["shared"] = rng.choice([1, 1, 2, 3, 4, 7, 8])
    case["n_new"] = rng.choice([1, 1, 1, 2, 3, 5])
    cap = 1 << 27  # key/value entries held, so that the plain form stays below the largest listed case
    case["max_len"] = _log_int(rng, 1, max(1, min(65536, cap // (case["B"] * case["kv_heads"] * dim))))
    return case


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split()]


def _lengths(case):
    """(length of each sequence with its new tokens, new tokens of each sequence): fixed by the case."""
    B, n, top = case["B"], case["n_new"], case["max_len"]
    if not case["ragged"]:
        return [max(top, n)] * B, [n] * B
    pick = random.Random(B * 1000003 + top * 31 + n)
    lens, news = [], []
    for b in range(B):
        new = n if n == 1 else pick.randint(0, n)
        length = max(new, int(top * pick.random() ** 2))
        if b == 0:
            length, new = max(top, n), n
        elif b == 1:
            length, new = new, new          # a first call: nothing cached before it
        elif b == 2:
            length, new = 0, 0              # an empty slot
        lens.append(length)
        news.append(new)
    return lens, news


# ------------------------------------------------------------------ layouts (include/ifq.h)
def _pack_tiles(n):
    """codes uint8 [R][C] (R % 16 == 0, C % 64 == 0) -> [R/16][C/64][512] bytes."""
    R, C = n.shape
    n = n.view(R // 16, 2, 8, C // 64, 2, 4, 8).permute(0, 3, 2, 5, 4, 1, 6)  # tile, ct, g, w, c, hi, code
    lo, hi = n[..., [0, 4, 1, 5]], n[..., [2, 6, 3, 7]]
    return (lo | (hi << 4)).reshape(R // 16, C // 64, 512)


def _unpack_tiles(t):
    """bytes [...][tile rows][ct][512] -> codes uint8 [...][16 tile rows][64 ct]."""
    lead, (RT, CT) = t.shape[:-3], t.shape[-3:-1]
    k = len(lead)
    b = t.reshape(*lead, RT, CT, 8, 4, 2, 2, 4)
    n = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)[..., WORD_PLACE]
    n = n.permute(*range(k), *(k + i for i in (0, 5, 2, 1, 4, 3, 6)))   # tile, hi, g, ct, c, w, code
    return n.reshape(*lead, RT * 16, CT * 64)


def _pack_scales(s):
    """bf16 [rows][groups] -> [ceil(rows/16)][groups][16], rows g and g + 8 of a tile side by side."""
    rows, ng = s.shape
    rt = (rows + 15) // 16
    full = torch.zeros(rt * 16, ng, dtype=s.dtype, device=s.device)
    full[:rows] = s
    return full.view(rt, 2, 8, ng).permute(0, 3, 2, 1).reshape(rt, ng, 16).contiguous()


def _unpack_scales(s, rows):
    rt, ng = s.shape[:2]
    return s.view(rt, ng, 8, 2).permute(0, 3, 2, 1).reshape(rt * 16, ng)[:rows]


# ------------------------------------------------------------------ plain forms: 4-bit layers
def _w4_codes(R, group):
    """Plain quantizer: codes q (float32, -7..7) and bf16 scales of float32 R [rows][cols]."""
    rows, cols = R.shape
    w = torch.where(torch.isfinite(R), R, torch.zeros_like(R)).view(rows, cols // group, group)
    s = (w.abs().amax(-1) / 7).to(torch.bfloat16)
    # the quotient next to a half needs more than 32 bits
    q = torch.round(w.double() / s.double().unsqueeze(-1))
    q = torch.where(s.unsqueeze(-1) == 0, torch.zeros_like(q), q).clamp(-7, 7)
    return q.float().view(rows, cols), s


def _w4_pack(R, group):
    rows, cols = R.shape
    rt = (rows + 15) // 16
    codes = torch.empty(rt, cols // 64, 512, dtype=torch.uint8, device=R.device)
    scales = torch.empty(rt, cols // group, 16, dtype=torch.bfloat16, device=R.device)
    step = 16 * max(1, (1 << 26) // (16 * cols))
    for r in range(0, rows, step):
        q, s = _w4_codes(R[r:r + step], group)
        n = torch.full((-(-q.shape[0] // 16) * 16, cols), 8, dtype=torch.uint8, device=R.device)
        n[:q.shape[0]] = (q + 8).to(torch.uint8)
        codes[r // 16:r // 16 + n.shape[0] // 16] = _pack_tiles(n)
        scales[r // 16:r // 16 + n.shape[0] // 16] = _pack_scales(s)
    return codes, scales


def _w4_values(codes, scales, rows, group):
    q = _unpack_tiles(codes)[:rows].float() - 8
    s = _unpack_scales(scales, rows).float()
    return (q.view(rows, -1, group) * s.unsqueeze(-1)).view(rows, -1)


def _plain_w4_quantize(st):
    R, group = st["R"], st["case"]["group"]
    codes, scales = _w4_pack(R, group)
    return _w4_values(codes, scales, R.shape[0], group).to(torch.bfloat16)


def _plain_w4_gemv(st):
    outs = []
    for d in st["layers"]:
        W = _w4_values(d["codes"], d["scales"], d["rows"], st["case"]["group"])
        x = d["x_re"] if d["x_im"] is None else torch.cat([d["x_re"], d["x_im"]], dim=1)
        y = x.float() @ W.t()
        if d["y_im"] is None:
            outs.append(y)
        else:
            half = d["rows"] // 2
            outs += [y[:, :half].contiguous(), y[:, half:].contiguous()]
    return outs


# ------------------------------------------------------------------ plain forms: 4-bit cache
def _kv_codes(x):
    """Plain quantizer of one plane: x float32 [..., dim] -> codes uint8, scale and minimum bf16 [...]."""
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).clamp(-BF16_MAX, BF16_MAX)
    lo, hi = x.amin(-1), x.amax(-1)
    m = lo.to(torch.bfloat16)
    s = (hi / 15 - lo / 15).to(torch.bfloat16)
    n = torch.round((x.double() - m.double().unsqueeze(-1)) / s.double().unsqueeze(-1))
    n = torch.where(s.unsqueeze(-1) == 0, torch.zeros_like(n), n).clamp(0, 15)
    return n.to(torch.uint8), s, m


def _kv_values(n, s, m):
    return s.float().unsqueeze(-1) * n.float() + m.float().unsqueeze(-1)


def _kv_pack_pages(k, v, dim, page):
    """k, v float32 [pages * page tokens][heads][2 dim] -> records [pages][heads][page/16][32 dim + 256]."""
    tok, H, D = k.shape
    T, ct = tok // 16, D // 64
    rec = torch.empty(H, T, 16 * D + 256, dtype=torch.uint8, device=k.device)
    for x, code_at, par_at in ((k, 0, 16 * D), (v, 8 * D, 16 * D + 128)):
        n, s, m = _kv_codes(x.view(tok, H, 2, dim))
        n = n.view(tok, H, D).permute(1, 0, 2)                                    # [H][tok][D]
        if code_at == 0:
            c = _pack_tiles(n.reshape(H * tok, D)).view(H, T, 8 * D)
        else:
            z = n.reshape(H, T, 2, 4, 2, ct, 2, 8, 4).permute(0, 1, 5, 7, 3, 6, 2, 4, 8)  # ct, g, t, qq, hi, e, i
            c = (z[..., 0::2] | (z[..., 1::2] << 4)).reshape(H, T, 8 * D)
        rec[:, :, code_at:code_at + 8 * D] = c
        par = torch.stack([s[..., 0], m[..., 0], s[..., 1], m[..., 1]], dim=-1)   # [tok][H][4]
        rec[:, :, par_at:par_at + 128] = par.permute(1, 0, 2).contiguous().view(torch.uint8).view(H, T, 128)
    return rec.view(H, tok // page, page // 16, -1).permute(1, 0, 2, 3).contiguous()


def _kv_unpack(rec, dim):
    """records [H][T][32 dim + 256] -> k, v float32 [H][16 T][2 dim]."""
    H, T, _ = rec.shape
    D = 2 * dim
    outs = []
    for code_at, par_at in ((0, 16 * D), (8 * D, 16 * D + 128)):
        c = rec[:, :, code_at:code_at + 8 * D]
        if code_at == 0:
            n = _unpack_tiles(c.reshape(H, T, 1, D // 64, 512)).view(H, T * 16, D)
        else:
            z = torch.stack([c & 15, c >> 4], dim=-1).view(H, T, D // 64, 8, 4, 2, 2, 2, 4)
            n = z.permute(0, 1, 6, 4, 7, 2, 5, 3, 8).reshape(H, T * 16, D)        # hi, t, e, ct, qq, g, i
        par = rec[:, :, par_at:par_at + 128].contiguous().view(torch.bfloat16).view(H, T * 16, 2, 2)
        outs.append(_kv_values(n.view(H, T * 16, 2, dim), par[..., 0], par[..., 1]).view(H, T * 16, D))
    return outs


def _plain_kv4_append(st):
    """Quantizes the new tokens into their places in the cache and returns the values they now stand for."""
    case, cache, table = st["case"], st["records"], st["page_table"]
    H, dim, page = case["kv_heads"], case["dim"], case["page"]
    D, flat, rec = 2 * dim, cache.view(-1), 32 * dim + 256
    outs = [torch.zeros_like(st[n]) for n in ("k_re", "k_im", "v_re", "v_im")]
    seq = torch.tensor([b for b, n in enumerate(st["news"]) for _ in range(n)], dtype=torch.int64, device=DEV)
    pos = torch.tensor([st["lens"][b] - n + i for b, n in enumerate(st["news"]) for i in range(n)],
                       dtype=torch.int64, device=DEV)
    rows = seq.numel()
    if rows == 0:
        return outs
    pg = table[seq, pos // page].long()
    tile = (pg[:, None] * H + torch.arange(H, device=DEV)) * (page // 16) + ((pos % page) // 16)[:, None]
    base, r = tile * rec, (pos % 16)[:, None]                                      # [rows][H], [rows][1]
    byte = torch.arange(D // 2, device=DEV)
    # byte f of a token's keys holds two codes of one word; of its values two entries of one half word
    ct, w, c, bb = byte // 32, (byte // 4) % 4, (byte // 16) % 2, byte % 4
    k_at = ct * 512 + ((r % 8) * 4 + w) * 16 + (c * 2 + r // 8) * 4 + bb
    k_lo = ct * 64 + c * 32 + w * 8 + torch.tensor([0, 4, 1, 5], device=DEV)[bb]
    q, g, ii = byte // 16, (byte // 2) % 8, byte % 2
    v_at = (q // 2) * 512 + (g * 4 + (r % 8) // 2) * 16 + ((q % 2) * 2 + r // 8) * 4 + (r % 2) * 2 + ii
    v_lo = q * 32 + g * 4 + 2 * ii
    for names, code_at, par_at, at, lo, step, oi in ((("k_re", "k_im"), 0, 16 * D, k_at, k_lo, 2, 0),
                                                     (("v_re", "v_im"), 8 * D, 16 * D + 128, v_at, v_lo, 1, 2)):
        x = torch.stack([st[n][:rows].view(rows, H, dim) for n in names], dim=2)
        n, s, m = _kv_codes(x)
        nf = n.view(rows, H, D)
        flat[(base + code_at)[:, :, None] + at[:, None, :]] = nf[..., lo] | (nf[..., lo + step] << 4)
        par = torch.stack([s[..., 0], m[..., 0], s[..., 1], m[..., 1]], dim=-1).contiguous().view(torch.uint8)
        flat[(base + par_at + r * 8)[:, :, None] + torch.arange(8, device=DEV)] = par
        val = _kv_values(n, s, m)
        outs[oi][:rows] = val[:, :, 0].reshape(rows, H * dim)
        outs[oi + 1][:rows] = val[:, :, 1].reshape(rows, H * dim)
    return outs


def _plain_kv4_attention(st):
    case, cache, table = st["case"], st["records"], st["page_table"]
    H, G, dim, page = case["kv_heads"], case["shared"], case["dim"], case["page"]
    outs = [torch.zeros_like(st["q_re"], dtype=torch.bfloat16) for _ in range(2)]
    row = 0
    for b, (length, new) in enumerate(zip(st["lens"], st["news"])):
        if new and length:
            pages = table[b, :-(-length // page)].long()
            rec = cache[pages].permute(1, 0, 2, 3).reshape(H, -1, 32 * dim + 256)
            k, v = (t[:, :length] for t in _kv_unpack(rec, dim))
            q = torch.cat([st[n][row:row + new].view(new, H, G, dim) for n in ("q_re", "q_im")], dim=-1)
            q = q.permute(1, 0, 2, 3).reshape(H, new * G, 2 * dim)
            s = (q @ k.transpose(1, 2)) * st["scale"]
            seen = torch.arange(length, device=DEV)[None, :] <= length - new + torch.arange(new, device=DEV)[:, None]
            s = s.masked_fill(~seen.repeat_interleave(G, 0), float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p @ v) / p.sum(-1, keepdim=True)
            o = o.view(H, new, G, 2, dim).permute(3, 1, 0, 2, 4).reshape(2, new, H * G * dim)
            outs[0][row:row + new] = o[0]
            outs[1][row:row + new] = o[1]
        row += new
    return outs


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed & 0x7FFFFFFF)
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _weights(rows, cols, g):
    """Weights as a trained layer has them: N(0, 0.02), every row with a gain of its own."""
    return 0.02 * _randn((rows, cols), g) * torch.exp(0.3 * _randn((rows, 1), g))


def _kv_plane(tokens, heads, dim, g, outlier):
    """Rotated keys (a few large entries per head) or values."""
    x = _randn((tokens, heads, dim), g)
    if outlier:
        x[..., ::max(1, dim // 4)] *= 6.0
    return x


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "w4_quantize":
        st["R"] = _weights(case["rows"], case["cols"], g)
        return st
    if op == "w4_gemv":
        st["layers"] = []
        for rows, cols in _shapes(case):
            codes, scales = _w4_pack(_weights(rows, cols, g), case["group"])
            d = {"codes": codes, "scales": scales, "rows": rows, "cols": cols}
            planes = 2 if case["planar"] else 1
            x = [_randn((case["B"], cols // planes), g, torch.bfloat16) for _ in range(planes)]
            y = [torch.empty(case["B"], rows // planes, device=DEV) for _ in range(planes)]
            d["x_re"], d["y_re"] = x[0], y[0]
            d["x_im"], d["y_im"] = (x[1], y[1]) if planes == 2 else (None, None)
            st["layers"].append(d)
        return st
    H, dim, page, B = case["kv_heads"], case["dim"], case["page"], case["B"]
    st["lens"], st["news"] = lens, news = _lengths(case)
    need = [-(-n // page) for n in lens]
    cols = max(1, max(need))
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st["page_table"] = table
    st["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    offs = [0]
    for n in news:
        offs.append(offs[-1] + n)
    st["new_offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV)
    rows = max(1, offs[-1])
    rec = torch.empty(pages, H, page // 16, 32 * dim + 256, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (page * H * 2 * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k = torch.cat([_kv_plane(n * page, H, dim, g, True) for _ in range(2)], dim=-1)
        v = torch.cat([_kv_plane(n * page, H, dim, g, False) for _ in range(2)], dim=-1)
        rec[p:p + n] = _kv_pack_pages(k, v, dim, page)
    st["records"] = rec
    if op == "kv4_append":
        for name in ("k_re", "k_im", "v_re", "v_im"):
            st[name] = _kv_plane(rows, H, dim, g, name[0] == "k").reshape(rows, H * dim)
    else:
        width = H * case["shared"] * dim
        st["q_re"], st["q_im"] = 1.5 * _randn((rows, width), g), 1.5 * _randn((rows, width), g)
        st["scale"] = 1.0 / math.sqrt(2 * dim)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if not own or case["op"] == "w4_gemv":
        return st
    import bit_complex_quantized_b200 as Q
    if case["op"] == "w4_quantize":
        rows, cols, rt = case["rows"], case["cols"], (case["rows"] + 15) // 16
        st["codes"] = torch.empty(rt, cols // 64, 512, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(rt, cols // case["group"], 16, dtype=torch.bfloat16, device=DEV)
        st["out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
        return st
    st["cache"] = Q.Kv4Cache(st["records"], st["page_table"], st["kv_lens"], case["dim"], n_new=case["n_new"],
                             rows=max(1, sum(st["news"])), new_offsets=st["new_offsets"])
    if case["op"] == "kv4_append":
        st["out"] = [torch.zeros_like(st[n]) for n in ("k_re", "k_im", "v_re", "v_im")]
    else:
        st["out"] = [torch.zeros_like(st["q_re"], dtype=torch.bfloat16) for _ in range(2)]
        nbytes = Q.ifq_kv4_attention_workspace_bytes(st["cache"], case["kv_heads"] * case["shared"])
        st["workspace"] = torch.empty(max(16, nbytes), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"w4_quantize": _plain_w4_quantize, "w4_gemv": _plain_w4_gemv, "kv4_append": _plain_kv4_append,
                "kv4_attention": _plain_kv4_attention}[op](state)
    import bit_complex_quantized_b200 as Q
    if op == "w4_quantize":
        group = state["case"]["group"]
        Q.ifq_w4_quantize([(state["R"], state["codes"], state["scales"])], group)
        Q.ifq_w4_dequantize([(state["codes"], state["scales"], state["out"])], group)
        return state["out"]
    if op == "w4_gemv":
        Q.ifq_w4_gemv(state["layers"], state["case"]["group"], state["case"]["B"])
        return [d[n] for d in state["layers"] for n in ("y_re", "y_im") if d[n] is not None]
    if op == "kv4_append":
        Q.ifq_kv4_append(state["cache"], *(state[n] for n in ("k_re", "k_im", "v_re", "v_im")))
        Q.ifq_kv4_read(state["cache"], *state["out"])
        return state["out"]
    Q.ifq_kv4_attention(state["cache"], state["q_re"], state["q_im"], *state["out"], scale=state["scale"],
                        workspace=state["workspace"])
    return state["out"]


# ------------------------------------------------------------------ work of one pass
def work(case):
    op = case["op"]
    if op == "w4_quantize":
        n, ng = case["rows"] * case["cols"], case["rows"] * case["cols"] // case["group"]
        # R once, codes and scales once, the values they stand for once
        return {"bytes": 4 * n + n // 2 + 2 * ng + 2 * n, "flops": 3 * n}
    if op == "w4_gemv":
        nbytes = flops = 0
        for r, c in _shapes(case):
            nbytes += r * c // 2 + 2 * r * c // case["group"] + case["B"] * (2 * c + 4 * r)
            flops += 2 * case["B"] * r * c
        return {"bytes": nbytes, "flops": flops}
    lens, news = _lengths(case)
    H, dim = case["kv_heads"], case["dim"]
    if op == "kv4_append":
        rows = sum(news)
        # k and v once, their records once, the values they stand for once
        return {"bytes": rows * H * (16 * dim + 2 * dim + 16 + 16 * dim), "flops": rows * H * 4 * dim * 6}
    Hq = H * case["shared"]
    seen = sum(n * (2 * (L - n) + n + 1) // 2 for L, n in zip(lens, news))
    held = sum(L for L, n in zip(lens, news) if n)
    return {"bytes": held * H * (2 * dim + 16) + sum(news) * Hq * dim * (8 + 4),
            "flops": seen * Hq * (2 * 2 * dim + 2 * 2 * dim + 4)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _entry_w4(codes, rows0, rows1, cols):
    """Codes of rows [rows0, rows1) by the address of each entry."""
    r = torch.arange(rows0, rows1, device=DEV)[:, None]
    c = torch.arange(cols, device=DEV)[None, :]
    byte = ((r // 16) * (cols // 64) + c // 64) * 512 + ((r % 8) * 4 + (c % 32) // 8) * 16
    byte = byte + (((c % 64) // 32) * 2 + (r % 16) // 8) * 4
    bit = ((c % 8) // 2) * 4 + (c % 2) * 16
    return ((codes.view(-1)[byte + bit // 8].to(torch.int32) >> (bit % 8)) & 15).double()


def _exact_w4_scale(scales, rows0, rows1, cols, group):
    r = torch.arange(rows0, rows1, device=DEV)[:, None]
    k = torch.arange(cols, device=DEV)[None, :] // group
    return scales.view(-1)[((r // 16) * (cols // group) + k) * 16 + 2 * (r % 8) + (r % 16) // 8].double()


def _exact_w4_quantize(st):
    R, group = st["R"], st["case"]["group"]
    out = []
    for r in range(0, R.shape[0], 1024):
        w = R[r:r + 1024]
        w = torch.nan_to_num(w, nan=0.0, posinf=0.0, neginf=0.0).unflatten(1, (-1, group))
        s = torch.div(w.abs().max(dim=2, keepdim=True).values, 7.0).bfloat16().double()
        ratio = torch.where(s > 0, w.double() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))
        out.append((ratio.round().clamp(-7, 7) * s).flatten(1))
    return torch.cat(out)


def _exact_w4_gemv(st):
    outs, group = [], st["case"]["group"]
    for d in st["layers"]:
        x = torch.cat([t.double() for t in (d["x_re"], d["x_im"]) if t is not None], dim=1)
        ys = []
        for r in range(0, d["rows"], 512):
            e = min(d["rows"], r + 512)
            w = (_entry_w4(d["codes"], r, e, d["cols"]) - 8) * _exact_w4_scale(d["scales"], r, e, d["cols"], group)
            ys.append(torch.einsum("bk,rk->br", x, w))
        y = torch.cat(ys, dim=1)
        outs += [y] if d["y_im"] is None else [y[:, :d["rows"] // 2], y[:, d["rows"] // 2:]]
    return outs


def _exact_kv4_append(st):
    case = st["case"]
    outs, rows = [], sum(st["news"])
    for name in ("k_re", "k_im", "v_re", "v_im"):
        x = torch.nan_to_num(st[name], nan=0.0, posinf=0.0, neginf=0.0).clamp(-BF16_MAX, BF16_MAX)
        x = x.unflatten(1, (case["kv_heads"], case["dim"]))
        lo, hi = x.min(dim=2, keepdim=True).values, x.max(dim=2, keepdim=True).values
        s = (torch.div(hi, 15.0) - torch.div(lo, 15.0)).bfloat16().double()
        m = lo.bfloat16().double()
        n = torch.where(s > 0, ((x.double() - m) / torch.where(s > 0, s, torch.ones_like(s))).round(),
                        torch.zeros_like(s)).clamp(0, 15)
        y = (n * s + m).flatten(1)
        y[rows:] = 0
        outs.append(y)
    return outs


def _exact_kv4_attention(st):
    case, cache = st["case"], st["records"].view(-1)
    H, G, dim, page = case["kv_heads"], case["shared"], case["dim"], case["page"]
    D, rec = 2 * dim, 32 * dim + 256
    outs = [torch.zeros(st["q_re"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
    d = torch.arange(D, device=DEV)[None, :]
    row = 0
    for b, (length, new) in enumerate(zip(st["lens"], st["news"])):
        if not new or not length:
            row += new
            continue
        t = torch.arange(length, device=DEV)
        pg = st["page_table"][b][t // page].long()
        r = (t % 16)[:, None]
        k_byte = (d // 64) * 512 + ((r % 8) * 4 + (d % 32) // 8) * 16 + (((d % 64) // 32) * 2 + r // 8) * 4
        k_bit = ((d % 8) // 2) * 4 + (d % 2) * 16 + 0 * r
        v_byte = (d // 64) * 512 + (((d % 32) // 4) * 4 + (r % 8) // 2) * 16 + (((d % 64) // 32) * 2 + r // 8) * 4
        v_bit = (d % 4) * 4 + (r % 2) * 16
        for h in range(H):
            base = (((pg * H + h) * (page // 16) + (t % page) // 16) * rec)[:, None]
            kv = []
            for code_at, par_at, byte, bit in ((0, 16 * D, k_byte, k_bit), (8 * D, 16 * D + 128, v_byte, v_bit)):
                n = (cache[base + code_at + byte + bit // 8].to(torch.int32) >> (bit % 8)) & 15
                par = cache[base + par_at + r * 8 + torch.arange(8, device=DEV)].view(torch.bfloat16).double()
                plane = torch.arange(D, device=DEV) // dim
                kv.append(n.double() * par[:, 2 * plane] + par[:, 2 * plane + 1])
            k, v = kv
            cols = slice(h * G * dim, (h + 1) * G * dim)
            q = torch.cat([st[n][row:row + new, cols].double().reshape(new * G, dim) for n in ("q_re", "q_im")], 1)
            s = torch.einsum("qd,td->qt", q, k) * st["scale"]
            last = (length - new + torch.arange(new, device=DEV)).repeat_interleave(G)
            s = torch.where(t[None, :] <= last[:, None], s, torch.full_like(s, -math.inf))
            o = torch.softmax(s, dim=1) @ v
            outs[0][row:row + new, cols] = o[:, :dim].reshape(new, G * dim)
            outs[1][row:row + new, cols] = o[:, dim:].reshape(new, G * dim)
        row += new
    return outs


def exact(case, seed):
    st = _inputs(case, seed)
    return {"w4_quantize": _exact_w4_quantize, "w4_gemv": _exact_w4_gemv, "kv4_append": _exact_kv4_append,
            "kv4_attention": _exact_kv4_attention}[case["op"]](st)
