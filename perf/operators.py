"""The operators by which a decoder reads the encoder's states, as cases that can be timed.

Four operators: rows or weights into 8-bit floating point with a power-of-two
scale per block of 128 ("quantize"), the product of two such matrices with the
quantisation of its activations ("linear"), attention of a decoder's tokens
over the encoder states of their clip ("cross"), and the attention weights of
chosen heads, which word timestamps are read from ("weights").

``run`` computes each in a plain form (elementary torch operations in 32 bits)
or, with ``own`` set, through this repository's entry points.
"""
import math

import torch

own = False

HEAD = 64
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # One decoder step of five beams through a 768-wide projection: all latency.
        {"name": "linear_step_5x768", "op": "linear", "M": 5, "N": 768, "K": 768, "x": "bf16", "epi": "bf16", "bias": True},
        # One 30 s clip (390 tokens) through the wide feed-forward product.
        {"name": "linear_clip_390x5120", "op": "linear", "M": 390, "N": 5120, "K": 1280, "x": "bf16", "epi": "bf16", "bias": True},
        # Sixteen 30 s clips through the narrow feed-forward product, added to the fp32 residual stream.
        {"name": "linear_fc2_6240", "op": "linear", "M": 6240, "N": 1280, "K": 5120, "x": "bf16", "epi": "resid", "bias": True},
        # Keys and values of all 12 decoder layers from the fp32 encoder output of 32 clips of 1500 frames.
        {"name": "linear_kv_48000", "op": "linear", "M": 48000, "N": 18432, "K": 768, "x": "f32", "epi": "bf16", "bias": True},
        # The feed-forward hidden rows of sixteen 30 s clips, one scale per row and 128 columns.
        {"name": "quantize_6240x5120", "op": "quantize", "M": 6240, "K": 5120, "x": "bf16", "rows": 1},
        # The adapter's gate and up weights when a checkpoint is loaded, one scale per 128 x 128 block.
        {"name": "quantize_weights_16384x2048", "op": "quantize", "M": 16384, "K": 2048, "x": "f32", "rows": 128},
        # One token of one clip's transcript over 1500 frames.
        {"name": "cross_step_1x1500", "op": "cross", "segs": 1, "tokens": 1, "states": 1500, "H": 12, "Hkv": 12,
         "dtype": "bf16", "layers": 1, "ragged": False},
        # Five beams of 32 clips, one token each, reading one layer's columns of the keys and values of all 12 layers.
        {"name": "cross_beams_32x5", "op": "cross", "segs": 32, "tokens": 5, "states": 1500, "H": 12, "Hkv": 12,
         "dtype": "bf16", "layers": 12, "ragged": False},
        # One token over the states of long recordings (up to 600 s) of four different lengths, grouped heads, f16.
        {"name": "cross_long_4x30000", "op": "cross", "segs": 4, "tokens": 1, "states": 30000, "H": 20, "Hkv": 4,
         "dtype": "f16", "layers": 1, "ragged": True},
        # Rescoring five hypotheses of 448 tokens for each of 32 clips.
        {"name": "cross_rescore_32x2240", "op": "cross", "segs": 32, "tokens": 2240, "states": 1500, "H": 12, "Hkv": 12,
         "dtype": "bf16", "layers": 1, "ragged": False},
        # The attention weights of one step, all 12 heads: what a timestamp decoder is handed per token.
        {"name": "weights_step_1x1500", "op": "weights", "segs": 1, "tokens": 1, "states": 1500, "H": 12, "Hkv": 12,
         "dtype": "bf16", "heads": 12, "ragged": False},
        # The alignment of whole transcripts: ten heads over 448 tokens of 32 clips.
        {"name": "weights_align_32x448", "op": "weights", "segs": 32, "tokens": 448, "states": 1500, "H": 12, "Hkv": 12,
         "dtype": "bf16", "heads": 10, "ragged": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "quantize", "cross", "cross", "cross", "weights"])
    if op == "linear":
        n, k = _log(rng, 64, 18432, 16), _log(rng, 64, 8192, 16)
        most = max(1, min(48000, 600_000_000_000 // (n * k), 800_000_000 // n))
        return {"op": op, "M": _log(rng, 1, most), "N": n, "K": k, "x": rng.choice(["bf16", "f16", "f32"]),
                "epi": rng.choice(["bf16", "bf16", "f16", "f32", "resid"]), "bias": rng.random() < 0.7}
    if op == "quantize":
        k = _log(rng, 16, 8192, 16)
        return {"op": op, "M": _log(rng, 1, min(48000, 64_000_000 // k)), "K": k,
                "x": rng.choice(["bf16", "f16", "f32"]), "rows": rng.choice([1, 1, 128])}
    h, hkv = rng.choice([(12, 12), (20, 20), (20, 4), (16, 8), (8, 1), (6, 2), (4, 4)])
    segs = _log(rng, 1, 32)
    states = _log(rng, 1, 30000)
    tokens = _log(rng, 1, 2240)
    case = {"op": op, "segs": segs, "tokens": tokens, "states": states, "H": h, "Hkv": hkv,
            "dtype": rng.choice(["bf16", "f16"])}
    if op == "cross":
        case["layers"] = rng.choice([1, 1, 4])
        cost = lambda: segs * h * tokens * states  # noqa: E731
        limit = 1_200_000_000
    else:
        case["heads"] = rng.randint(1, h)
        cost = lambda: segs * h * tokens * states  # noqa: E731
        limit = 200_000_000
    while cost() > limit:  # shorten the longer axis until the case costs no more than the largest listed
        if tokens * 8 > states:
            tokens = max(1, tokens // 2)
        else:
            states = max(1, states // 2)
    case.update(tokens=tokens, states=states, ragged=rng.random() < 0.7)
    return case


def _lengths(n, most, ragged, odd):
    """Length of each segment: all alike, or spread from 1 to the longest."""
    if not ragged:
        return [most] * n
    return [most] + [1 + (i * odd + i * i) % most for i in range(1, n)]


def _segments(case):
    lq = _lengths(case["segs"], case["tokens"], case["ragged"], 7919)
    lk = _lengths(case["segs"], case["states"], case["ragged"], 10007)
    return lq, lk


# ------------------------------------------------------------------ plain forms

def _to_fp8(x, rows):
    """Codes and exponents of x with one power-of-two scale per `rows` x 128 block: the smallest scale whose
    448 reaches the block's largest magnitude."""
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // BLOCK)
    wide = torch.zeros((mb * rows, kb * BLOCK), dtype=torch.float32, device=x.device)
    wide[:m, :k] = x
    amax = wide.view(mb, rows, kb, BLOCK).abs().amax(dim=(1, 3))
    mant, e = torch.frexp(amax)                     # amax = mant 2^e, mant in [0.5, 1); 448 = 0.875 * 2^9
    s = (e - 9 + (mant > 0.875).int()).clamp(-127, 127)
    s = torch.where(amax == 0, torch.zeros_like(s), s)
    up = torch.ldexp(torch.ones_like(amax), -s).repeat_interleave(rows, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return (x.float() * up).to(torch.float8_e4m3fn), s


def _values(codes, s, rows):
    m, k = codes.shape
    scale = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s)
    return codes.float() * scale.repeat_interleave(rows, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]


def _scale_bytes(s):
    return (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _padded(x, cu, longest, heads):
    """Packed rows [T, heads * 64] as [segments, longest, heads, 64] in 32 bits, and which of them are real."""
    at = torch.arange(longest, device=x.device)[None] + cu[:-1, None].long()
    real = at < cu[1:, None]
    rows = x[at.clamp(max=max(x.shape[0] - 1, 0))].float()
    return rows.reshape(cu.numel() - 1, longest, heads, HEAD), real


def _probabilities(q, k, cu_q, cu_k, max_q, max_k, h, hkv):
    """[segments, h, max_q, max_k]: softmax over the segment's states of q . k / 8; zero without states."""
    qp, _ = _padded(q, cu_q, max_q, h)
    kp, real = _padded(k, cu_k, max_k, hkv)
    kp = kp.repeat_interleave(h // hkv, 2)
    s = (qp.permute(0, 2, 1, 3) @ kp.permute(0, 2, 3, 1)) * 0.125
    s = s.masked_fill(~real[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _packed(cu, t):
    """Segment and place within it of each packed row."""
    row = torch.arange(t, device=cu.device)
    seg = torch.searchsorted(cu, row.int(), right=True) - 1
    return seg, row - cu[seg]


# ------------------------------------------------------------------ cases

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def activations(m, k, dtype):
        # rows of different size with a few wide channels, as after a feed-forward activation
        x = normal(m, k) * torch.exp(normal(m, 1, std=0.5))
        x[:, :: 97] *= 8
        return x.to(dtype)

    st = {"op": op, "ws": torch.zeros(256, dtype=torch.uint8, device="cuda")}
    if op == "quantize":
        st["rows"] = case["rows"]
        st["x"] = (normal(case["M"], case["K"], std=0.02, dtype=DTYPES[case["x"]]) if case["rows"] > 1
                   else activations(case["M"], case["K"], DTYPES[case["x"]]))
    elif op == "linear":
        m, n, k = case["M"], case["N"], case["K"]
        codes, s = _to_fp8(normal(n, k, std=0.04), BLOCK)
        st.update(x=activations(m, k, DTYPES[case["x"]]), w=codes, ws_=_scale_bytes(s), s=s, epi=case["epi"],
                  bias=normal(n) if case["bias"] else None, out=normal(m, n) if case["epi"] == "resid" else None)
    else:
        lq, lk = _segments(case)
        h, hkv, dt, layers = case["H"], case["Hkv"], DTYPES[case["dtype"]], case.get("layers", 1)
        cu = lambda v: torch.tensor([0] + torch.tensor(v).cumsum(0).tolist(), dtype=torch.int32, device="cuda")  # noqa: E731
        wide = torch.empty((sum(lk), layers * 2 * hkv * HEAD), dtype=dt, device="cuda")
        at = (layers - 1) * 2 * hkv * HEAD  # the last layer's columns: keys, then values
        wide[:, at:] = normal(sum(lk), 2 * hkv * HEAD, dtype=dt)
        st.update(q=normal(sum(lq), h * HEAD, std=2.0, dtype=dt), k=wide[:, at:at + hkv * HEAD],
                  v=wide[:, at + hkv * HEAD:], cu_q=cu(lq), cu_k=cu(lk), max_q=max(lq), max_k=max(lk), h=h, hkv=hkv)
        if op == "weights":
            st["heads"] = torch.randperm(h, generator=g, device="cuda")[:case["heads"]].sort().values.int()
    return st


def run(st):
    op = st["op"]
    if own:
        import speech_recognition_audio_b200 as sra
        if op == "quantize":
            return sra.quantize_fp8(st["x"], st["rows"])
        if op == "linear":
            epi = {"bf16": sra.EPI_BF16, "f16": sra.EPI_F16, "f32": sra.EPI_F32, "resid": sra.EPI_F32_RESID}[st["epi"]]
            codes, scales = sra.quantize_fp8(st["x"])
            return sra.linear_fp8(codes, scales, st["w"], st["ws_"], st["bias"], epi, out=st["out"], workspace=st["ws"])
        if op == "cross":
            return sra.cross_attention(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["max_q"], st["max_k"],
                                       workspace=st["ws"], check=False)
        return sra.cross_attention_weights(st["q"], st["k"], st["cu_q"], st["cu_k"], st["max_q"], st["max_k"],
                                           heads=st["heads"], workspace=st["ws"], check=False)
    if op == "quantize":
        codes, s = _to_fp8(st["x"], st["rows"])
        return codes, _scale_bytes(s)
    if op == "linear":
        y = _values(*_to_fp8(st["x"], 1), 1) @ _values(st["w"], st["s"], BLOCK).t()
        if st["bias"] is not None:
            y += st["bias"]
        if st["out"] is not None:
            st["out"] += y
            return st["out"]
        return y.to(DTYPES[st["epi"]])
    p = _probabilities(st["q"], st["k"], st["cu_q"], st["cu_k"], st["max_q"], st["max_k"], st["h"], st["hkv"])
    seg, at = _packed(st["cu_q"], st["q"].shape[0])
    if op == "weights":
        return p[:, st["heads"].long()].permute(1, 0, 2, 3)[:, seg, at].contiguous()
    v, _ = _padded(st["v"], st["cu_k"], st["max_k"], st["hkv"])
    o = p @ v.repeat_interleave(st["h"] // st["hkv"], 2).permute(0, 2, 1, 3)
    return o.permute(0, 2, 1, 3)[seg, at].reshape(st["q"].shape).to(st["q"].dtype)


def work(case):
    op = case["op"]
    if op in ("quantize", "linear"):
        m, k = case["M"], case["K"]
        x = m * k * (4 if case["x"] == "f32" else 2)
        kb = -(-k // BLOCK)
        if op == "quantize":
            return {"bytes": x + m * k + -(-m // case["rows"]) * kb, "flops": 2 * m * k}
        n = case["N"]
        y = m * n * {"bf16": 2, "f16": 2, "f32": 4, "resid": 8}[case["epi"]]
        return {"bytes": x + n * k + -(-n // BLOCK) * kb + (4 * n if case["bias"] else 0) + y, "flops": 2 * m * n * k}
    lq, lk = _segments(case)
    h, hkv = case["H"], case["Hkv"]
    pairs = sum(a * b for a, b in zip(lq, lk))
    if op == "cross":
        return {"bytes": 2 * HEAD * (2 * h * sum(lq) + 2 * hkv * sum(lk)), "flops": 4 * HEAD * h * pairs}
    n = case["heads"]
    return {"bytes": 2 * HEAD * (n * sum(lq) + min(n, hkv) * sum(lk)) + 4 * n * sum(lq) * max(lk), "flops": 2 * HEAD * n * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def _grid8(x):
    """x rounded to the nearest value with 4 significant bits (exponents from -6, ties to even), from the definition."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    e = e - (x.abs() < torch.exp2(e)).double() * (e > -6).double() + (x.abs() >= torch.exp2(e + 1)).double()
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _blocks64(x, rows):
    """Values of x on the grid, as multiples of the block's scale, and that scale, block row by block row."""
    m, k = x.shape
    codes = torch.empty((m, k), dtype=torch.float64, device=x.device)
    scale = torch.empty((-(-m // rows), -(-k // BLOCK)), dtype=torch.float64, device=x.device)
    for j in range(scale.shape[1]):
        c = x[:, j * BLOCK:(j + 1) * BLOCK].double()
        top = c.abs().amax(1)
        if rows > 1:
            top = torch.nn.functional.pad(top, (0, scale.shape[0] * rows - m)).view(-1, rows).amax(1)
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(-127, 127)
        e = e + (448 * torch.exp2(e) < top).double() - (448 * torch.exp2(e - 1) >= top).double() * (e > -127).double()
        scale[:, j] = torch.where(top == 0, torch.ones_like(e), torch.exp2(e))
        codes[:, j * BLOCK:(j + 1) * BLOCK] = _grid8(c / scale[:, j].repeat_interleave(rows)[:m, None])
    return codes, scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _blocks64(st["x"], case["rows"])
    if op == "linear":
        codes, scale = _blocks64(st["x"], 1)
        x = codes * scale.repeat_interleave(BLOCK, 1)[:, :case["K"]]
        w = st["w"].double()
        for j in range(st["s"].shape[1]):
            w[:, j * BLOCK:(j + 1) * BLOCK] *= torch.exp2(st["s"][:, j].double()).repeat_interleave(BLOCK)[:case["N"], None]
        y = x @ w.t()
        if st["bias"] is not None:
            y += st["bias"].double()
        return y if st["out"] is None else y + st["out"].double()
    lq, lk = _segments(case)
    h, group = case["H"], case["H"] // case["Hkv"]
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    w = None
    if op == "weights":
        w = torch.zeros((case["heads"], q.shape[0], max(lk)), dtype=torch.float64, device="cuda")
    picked = st["heads"].tolist() if op == "weights" else range(h)
    r = c = 0
    for a, b in zip(lq, lk):
        for i, n in enumerate(picked):
            kv = slice(n // group * HEAD, n // group * HEAD + HEAD)
            p = torch.softmax(q[r:r + a, n * HEAD:(n + 1) * HEAD] @ k[c:c + b, kv].t() / 8, -1)
            if op == "weights":
                w[i, r:r + a, :b] = p
            else:
                out[r:r + a, n * HEAD:(n + 1) * HEAD] = p @ v[c:c + b, kv]
        r, c = r + a, c + b
    return w if op == "weights" else out
