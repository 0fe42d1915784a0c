"""The operators of few token rows, as they are measured: a residual RMS norm
whose output is MX-FP8 codes, and products of a few rows with a prepared 4-bit
weight, for rows in bf16 or fp32 and for rows already coded in MX-FP8.

  norm    h = x + residual, rounded to the stream's type;
          v = h / sqrt(mean(h^2) + eps) * gain;
          codes and scales of v: E4M3 elements, one power-of-two scale for
          each 32 (or 64) consecutive channels, the smallest 2^e with
          max|v| <= 448 * 2^e (the scale of 64 channels stands at both of its
          32-channel places)
  rows    y = x W + (x L1) L2, W held as E2M1 codes with one power-of-two
          scale for each 32 input channels of an output channel
  rows8   the same for x held as E4M3 codes with scales, as the norm gives them
  block   norm, then its codes through two such products (the query
          projection, and the key and value projections stacked)
"""
import math

import torch

own = False

EPS = 1e-6
GRID4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)          # the magnitudes of E2M1


def _norm(name, rows, channels, dtype="bf16", residual=True, group=32, plain=False, sliced=False):
    return dict(name=name, op="norm", rows=rows, channels=channels, dtype=dtype, residual=residual, group=group,
                plain=plain, sliced=sliced)


def _rows(name, rows, ci, co, rank=32, x="bf16", y="f32", sliced=False):
    return dict(name=name, op="rows", rows=rows, ci=ci, co=co, rank=rank, x=x, y=y, sliced=sliced)


def _rows8(name, rows, ci, co, rank=32, y="f32"):
    return dict(name=name, op="rows8", rows=rows, ci=ci, co=co, rank=rank, y=y)


def listed():
    return [
        # one token's residual stream between two layers of width 5120: latency
        _norm("norm_1x5120", 1, 5120),
        # two prompts of 512 text tokens; the norm's plain values are kept too, for a branch in 16 bits
        _norm("norm_1024x5120_plain", 1024, 5120, plain=True),
        # the Wan 1.3B grid's tokens in fp32, the first norm of a block (nothing to add), one scale for 64 channels
        _norm("norm_32760x1536_f32_g64", 32760, 1536, dtype="f32", residual=False, group=64),
        # the 720p grid's tokens at width 5120: the largest
        _norm("norm_75600x5120", 75600, 5120),
        # the smallest product: one row through the Wan 1.3B projection
        _rows("rows_1_1536to1536", 1, 1536, 1536),
        # two timestep vectors (a guidance pair) through a projection to six modulation vectors, fp32, no low-rank branch
        _rows("rows_2_5120to30720_f32", 2, 5120, 30720, rank=0, x="f32"),
        # sixteen rows through the FFN's second layer, an odd row stride of a wider buffer
        _rows("rows_16_13824to5120", 16, 13824, 5120, y="bf16", sliced=True),
        # an odd number of rows and of output channels, a narrow rank
        _rows("rows_37_2080to4999", 37, 2080, 4999, rank=16),
        # one coded row through the FFN's first layer
        _rows8("rows8_1_5120to13824", 1, 5120, 13824),
        # the most rows that count as few, coded, through the attention projection
        _rows8("rows8_64_5120to5120", 64, 5120, 5120, y="bf16"),
        # a decoding step of eight sequences: norm, query, stacked key and value
        dict(name="block_8x5120", op="block", rows=8, channels=5120, rank=32),
        # one sequence at the small width
        dict(name="block_1x1536", op="block", rows=1, channels=1536, rank=32),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "rows", "rows", "rows8", "rows8", "block"))
    if op == "norm":
        channels = 64 * _log_uniform(rng, 1, 216)
        most = 75600 * 5120 * 7 // (13 * channels)          # (fp32 rows move up to 13 bytes an element, bf16 ones 7)
        return dict(op="norm", rows=_log_uniform(rng, 1, min(75600, most)), channels=channels,
                    dtype=rng.choice(("bf16", "f32")), residual=rng.random() < 0.7, group=rng.choice((32, 64)),
                    plain=rng.random() < 0.3, sliced=rng.random() < 0.3)
    rows = _log_uniform(rng, 1, 64)
    rank = rng.choice((0, 8, 16, 32, 32, 48, 64, 128))
    if op == "block":
        return dict(op="block", rows=rows, channels=32 * _log_uniform(rng, 8, 160), rank=rank)
    ci = 32 * _log_uniform(rng, 8, 432)
    co = _log_uniform(rng, 128, min(30720, 13824 * 5120 // ci))
    y = rng.choice(("f32", "bf16"))
    if op == "rows8":
        return dict(op="rows8", rows=rows, ci=ci, co=co, rank=min(rank, ci, co), y=y)
    return dict(op="rows", rows=rows, ci=ci, co=co, rank=min(rank, ci, co), x=rng.choice(("bf16", "bf16", "f32")), y=y,
                sliced=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs ----
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, rows, channels, dtype, sliced=False):
    """Activations: channels of unequal size, a few of them large; `sliced`: a view into rows of a wider buffer."""
    wide = channels + (64 if sliced else 0)
    size = torch.exp(0.5 * _randn(g, wide))
    size[torch.randint(0, wide, (max(1, wide // 512),), generator=g, device="cuda")] *= 30.0
    x = torch.empty(rows, wide, dtype=TYPES[dtype], device="cuda")
    for i in range(0, rows, 8192):
        x[i:i + 8192] = (_randn(g, min(8192, rows - i), wide) * size).to(TYPES[dtype])
    return x[:, 32:32 + channels] if sliced else x


def _power(e):
    """2^e in fp32, built from its bits (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(largest, low, top):
    """The smallest e >= -126 with largest <= low * 2^(e + top), low in [1, 2)."""
    m, e = torch.frexp(largest)
    e = e - 1 - top + (2 * m > low).to(torch.int32)
    return torch.where(largest > 0, e, torch.full_like(e, -126)).clamp_min(-126)


def _weight(g, ci, co, rank):
    """A weight in hand: E2M1 codes (two to a byte, the even channel low) and E8M0 scale codes of a Gaussian residual, and its bf16 factors."""
    codes = torch.empty(co, ci // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(co, ci // 32, dtype=torch.uint8, device="cuda")
    middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for i in range(0, co, 4096):
        w = (_randn(g, min(4096, co - i), ci) / math.sqrt(ci)).view(-1, ci // 32, 32)
        e = _exponent(w.abs().amax(-1), 1.5, 2)
        u = w * _power(-e)[..., None]
        c = torch.bucketize(u.abs(), middle, out_int32=True) + 8 * (u < 0)
        c = c.view(-1, ci // 2, 2).to(torch.uint8)
        codes[i:i + 4096] = c[..., 0] | (c[..., 1] << 4)
        scales[i:i + 4096] = (e + 127).to(torch.uint8)
    l1 = (_randn(g, ci, rank) * ci ** -0.5).to(torch.bfloat16)
    l2 = _randn(g, rank, co).mul_(0.3).to(torch.bfloat16)
    return dict(codes=codes, scales=scales, l1=l1, l2=l2)


def _handle(w, rows):
    """The prepared weight of a program that loads 4-bit weights, and its workspace for up to `rows` rows."""
    from w4a4_quantized_linear_cube_amd import dq
    host = {k: v.cpu() for k, v in w.items()}
    bits = {k: host[k].view(torch.int16).numpy().view("uint16") if host[k].numel() else None for k in ("l1", "l2")}
    handle = dq.dq_import_weights(host["codes"].numpy(), host["scales"].numpy(), bits["l1"], bits["l2"], device=0)
    return dict(handle=handle, rows=dq.dq_rows_create(handle, rows))


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] in ("norm", "block"):
        n, c = case["rows"], case["channels"]
        dtype = case.get("dtype", "bf16")
        s["x"] = _tokens(g, n, c, dtype, case.get("sliced", False))
        s["residual"] = 2.0 * _tokens(g, n, c, dtype) if case.get("residual", True) else None
        s["gain"] = 1.0 + 0.2 * _randn(g, c)
        if own:
            s["h"] = torch.empty(n, c, dtype=TYPES[dtype], device="cuda") if s["residual"] is not None else None
            s["codes"] = torch.empty(n, c, dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.empty(n, c // 32, dtype=torch.float8_e8m0fnu, device="cuda")
            s["plain"] = torch.empty(n, c, dtype=TYPES[dtype], device="cuda") if case.get("plain") else None
    if case["op"] == "block":
        s["weights"] = [_weight(g, c, co, case["rank"]) for co in (c, 2 * c)]
        if own:
            s["weights"] = [_handle(w, n) for w in s["weights"]]
            s["y"] = [torch.empty(n, co, dtype=torch.bfloat16, device="cuda") for co in (c, 2 * c)]
    if case["op"] in ("rows", "rows8"):
        n, ci, co = case["rows"], case["ci"], case["co"]
        w = _weight(g, ci, co, case["rank"])
        if case["op"] == "rows":
            s["x"] = _tokens(g, n, ci, case["x"], case["sliced"])
        else:
            s["codes"], s["scales"] = _mx8(_tokens(g, n, ci, "f32"), 32)
        s["weights"] = [_handle(w, n) if own else w]
        if own:
            s["y"] = [torch.empty(n, co, dtype=TYPES[case["y"]], device="cuda")]
    return s


# ------------------------------------------------------------- plain forms ----
def _mx8(v, group):
    """fp32 rows to E4M3 elements and E8M0 scales."""
    u = v.view(v.shape[0], -1, group)
    e = _exponent(u.abs().amax(-1), 1.75, 8)
    codes = (u * _power(-e)[..., None]).view(v.shape).to(torch.float8_e4m3fn)
    scales = (e + 127).to(torch.uint8).repeat_interleave(group // 32, dim=1)
    return codes, scales.view(torch.float8_e8m0fnu)


def _plain_norm(s):
    x = s["x"]
    h = x
    if s["residual"] is not None:
        h = (x.float() + s["residual"].float()).to(x.dtype)
    # the statistics in 64 bits: an element next to the border of two codes goes by the last bit of the row's factor
    mean = h.double().square_().mean(-1, keepdim=True)
    factor = torch.rsqrt(mean + EPS).float()
    v = h.float() * factor * s["gain"]
    codes, scales = _mx8(v, s["case"].get("group", 32))
    out = dict(codes=codes, scales=scales)
    if s["residual"] is not None:
        out["h"] = h
    if s["case"].get("plain"):
        out["plain"] = v.to(x.dtype)
    return out


def _plain_product(x, w, dtype):
    """x fp32 [n][ci]; the weight decoded by a table, channel pairs side by side."""
    table = torch.tensor(GRID4 + tuple(-m for m in GRID4), device="cuda")
    co, half = w["codes"].shape
    dense = torch.stack((table[(w["codes"] & 15).int()], table[(w["codes"] >> 4).int()]), dim=-1)
    dense = (dense.view(co, half // 16, 32) * _power(w["scales"].int() - 127)[..., None]).view(co, 2 * half)
    y = x @ dense.t()
    if w["l1"].shape[1]:
        y += (x @ w["l1"].float()) @ w["l2"].float()
    return y.to(dtype)


def _values(codes, scales):
    """The fp32 values that E4M3 elements with their scales stand for."""
    n, c = codes.shape
    return (codes.float().view(n, c // 32, 32) * scales.float()[..., None]).view(n, c)


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "rows":
        return _plain_product(s["x"].float(), s["weights"][0], TYPES[case["y"]])
    if case["op"] == "rows8":
        return _plain_product(_values(s["codes"], s["scales"]), s["weights"][0], TYPES[case["y"]])
    out = _plain_norm(s)
    x = _values(out["codes"], out["scales"])
    out["q"] = _plain_product(x, s["weights"][0], torch.bfloat16)
    out["kv"] = _plain_product(x, s["weights"][1], torch.bfloat16)
    return out


def _run_own(s, case):
    from w4a4_quantized_linear_cube_amd import dq
    if case["op"] == "rows":
        w = s["weights"][0]
        dq.dq_linear_rows(w["handle"], s["x"], w["rows"], s["y"][0])
        return s["y"][0]
    if case["op"] == "rows8":
        w = s["weights"][0]
        dq.dq_linear_rows8(w["handle"], s["codes"], s["scales"], w["rows"], s["y"][0])
        return s["y"][0]
    group = case.get("group", 32)
    plain = s["plain"]
    dq.dq_rmsnorm8(s["x"], s["gain"], EPS, s["codes"], s["scales"], residual=s["residual"], h=s["h"], y=plain, group=group)
    out = dict(codes=s["codes"], scales=s["scales"])
    if s["h"] is not None:
        out["h"] = s["h"]
    if plain is not None:
        out["plain"] = plain
    if case["op"] == "block":
        for name, w, y in zip(("q", "kv"), s["weights"], s["y"]):
            dq.dq_linear_rows8(w["handle"], s["codes"], s["scales"], w["rows"], y)
            out[name] = y
    return out


def _product_work(n, ci, co, rank, x_bytes, y_bytes):
    factors = (ci + co) * rank
    return (ci * co / 2 + ci * co / 32 + 2 * factors + n * ci * x_bytes + n * co * y_bytes,
            2 * n * (ci * co + factors))


def work(case):
    n = case["rows"]
    size = {"bf16": 2, "f32": 4}
    nbytes = flops = 0
    if case["op"] in ("norm", "block"):
        c, e = case["channels"], size[case.get("dtype", "bf16")]
        streams = 1 + 2 * case.get("residual", True) + case.get("plain", False)
        nbytes += n * c * (streams * e + 1 + 1 / 32) + 4 * c
        flops += 5 * n * c
    coded = 1 + 1 / 32
    if case["op"] == "rows":
        products = [_product_work(n, case["ci"], case["co"], case["rank"], size[case["x"]], size[case["y"]])]
    elif case["op"] == "rows8":
        products = [_product_work(n, case["ci"], case["co"], case["rank"], coded, size[case["y"]])]
    elif case["op"] == "block":
        products = [_product_work(n, c, co, case["rank"], coded, 2) for co in (c, 2 * c)]
    else:
        products = []
    return dict(bytes=nbytes + sum(b for b, _ in products), flops=flops + sum(f for _, f in products))


# ----------------------------------------------------------------- in 64 bits ----
def _exact_element(byte, bits, mantissa):
    """The value of a small float from its fields: sign, exponent, mantissa."""
    byte = byte.to(torch.int32)
    sign = 1.0 - 2.0 * ((byte >> (bits - 1)) & 1).double()
    field = (byte >> mantissa) & ((1 << (bits - 1 - mantissa)) - 1)
    fraction = (byte & ((1 << mantissa) - 1)).double() / (1 << mantissa)
    bias = (1 << (bits - 2 - mantissa)) - 1
    exponent = field.clamp_min(1) - bias
    return sign * torch.ldexp(fraction + (field > 0).double(), exponent.double())


def _exact_norm(s):
    x = s["x"].double()
    out, h = {}, x
    if s["residual"] is not None:
        out["h"] = x + s["residual"].double()
        h = out["h"].to(s["x"].dtype).double()              # (the norm is that of the stream as it is stored)
    v = h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS) * s["gain"].double()
    if s["case"].get("plain"):
        out["plain"] = v
    n, c, group = v.shape[0], v.shape[1], s["case"].get("group", 32)
    u = v.view(n, c // group, group)
    e = torch.ceil(torch.log2(u.abs().amax(-1) / 448.0)).clamp_min(-126)
    u = u * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)
    out["codes"] = (torch.round(u / step) * step).view(n, c)
    out["scales"] = torch.exp2(e).repeat_interleave(group // 32, dim=1)
    return out


def _exact_product(x, w):
    co, half = w["codes"].shape
    dense = torch.empty(co, 2 * half, dtype=torch.float64, device="cuda")
    dense[:, 0::2] = _exact_element(w["codes"] & 15, 4, 1)
    dense[:, 1::2] = _exact_element(w["codes"] >> 4, 4, 1)
    dense *= torch.exp2(w["scales"].double() - 127).repeat_interleave(32, dim=1)
    return x @ dense.t() + x @ w["l1"].double() @ w["l2"].double()


def exact(case, seed):
    global own
    asked, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = asked
    if case["op"] == "rows":
        return _exact_product(s["x"].double(), s["weights"][0])
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "rows8":
        codes, scales = s["codes"], s["scales"].view(torch.uint8).double() - 127
        x = _exact_element(codes.view(torch.uint8), 8, 3) * torch.exp2(scales).repeat_interleave(32, dim=1)
        return _exact_product(x, s["weights"][0])
    out = _exact_norm(s)
    x = out["codes"] * out["scales"].repeat_interleave(32, dim=1)
    out["q"], out["kv"] = (_exact_product(x, w) for w in s["weights"])
    return out
