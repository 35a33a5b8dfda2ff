"""Measured cases of the layer's few-bit operators, with their plain forms.

Five operators around the MLA attention: the root-mean-square norm with the
residual's addition and an 8-bit output (``norm``), the projections with 4-bit
weights for bf16 or 8-bit activations (``linear``), the weights' way into that
format and back (``weights``), and the FP8 latent cache read back into bf16
pages (``read``).

Formats.  4-bit weights: ``w4`` [N, K/2] bytes, column 2i of a row in the low
half of byte i, column 2i + 1 in the high half; a value is ``(nibble - 8) *
scale[n, k // 128]`` with bf16 scales [N, ceil(K/128)].  8-bit activations: E4M3
codes [T, D] with one float32 scale for each 128 columns of a row.  FP8 cache:
E4M3 codes [P, 64, 512], float32 scale per token, f16 keys [P, 64, 64] that carry
1/scale.
"""

import math

import torch

own = False

GROUP = 128        # columns that share a scale
EPS = 1e-6
FLOOR = 2.0 ** -100  # smallest scale of an 8-bit group: an all-zero group divides by it
LATENT, ROPE, PAGE = 512, 64, 64
MOST = 16384 * 7168  # elements of the largest activation and of the largest weight


def listed():
    return [
        # one sequence decodes: the hidden state (7168) joins the residual stream before the attention
        {"name": "norm_t1_d7168_res", "op": "norm", "T": 1, "D": 7168, "residual": True, "fp8": False},
        # 32 sequences decode: the query's latent (1536) on its way into 8-bit projections
        {"name": "norm_t32_d1536_fp8", "op": "norm", "T": 32, "D": 1536, "residual": False, "fp8": True},
        # 8 prompts of 2048 tokens: the whole chunk's hidden state, 8 bits out
        {"name": "norm_t16384_d7168_res_fp8", "op": "norm", "T": 16384, "D": 7168, "residual": True, "fp8": True},
        # one sequence decodes: the hidden state to the query's latent
        {"name": "linear_t1_k7168_n1536", "op": "linear", "T": 1, "K": 7168, "N": 1536, "fp8": False},
        # a few sequences, the latent and its key side by side with one row more: ragged in every direction
        {"name": "linear_t5_k7104_n577_fp8", "op": "linear", "T": 5, "K": 7104, "N": 577, "fp8": True},
        # 32 sequences decode: the query's latent to all heads, 8-bit activations
        {"name": "linear_t32_k1536_n16384_fp8", "op": "linear", "T": 32, "K": 1536, "N": 16384, "fp8": True},
        # 64 sequences with 4 new tokens each: the output projection
        {"name": "linear_t256_k16384_n7168", "op": "linear", "T": 256, "K": 16384, "N": 7168, "fp8": False},
        # loading a layer: the smallest projection (the shared key) and the largest (the output)
        {"name": "weights_n64_k7168", "op": "weights", "N": 64, "K": 7168},
        {"name": "weights_n7168_k16384", "op": "weights", "N": 7168, "K": 16384},
        # a short prompt's cache before its next chunk
        {"name": "read_b1_l300", "op": "read", "B": 1, "lo": 300, "hi": 300},
        # the batched decode's cache
        {"name": "read_b32_l4096", "op": "read", "B": 32, "lo": 4096, "hi": 4096},
        # the ragged decode's cache
        {"name": "read_b128_l1024_8192", "op": "read", "B": 128, "lo": 1024, "hi": 8192},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "weights", "read"])
    if op == "norm":
        d = 8 * _spread(rng, 8, 2048)
        return {"op": op, "T": _spread(rng, 1, min(16384, MOST // d)), "D": d, "residual": rng.random() < 0.5,
                "fp8": rng.random() < 0.5}
    if op in ("linear", "weights"):
        k = 64 * _spread(rng, 1, 256)
        n = _spread(rng, 1, min(16384, MOST // k))
        if op == "weights":
            return {"op": op, "N": n, "K": k}
        return {"op": op, "T": _spread(rng, 1, 256), "K": k, "N": n, "fp8": rng.random() < 0.5}
    hi = _spread(rng, 1, 8192)
    return {"op": op, "B": _spread(rng, 1, 128), "lo": rng.randint(0, min(hi, 1024)), "hi": hi}


def _lengths(case):
    b = case["B"]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, b - 1) if i else case["hi"] for i in range(b)]


def work(case):
    op = case["op"]
    if op == "norm":
        t, d = case["T"], case["D"]
        out = t * d + 4 * t * -(-d // GROUP) if case["fp8"] else 2 * t * d
        return {"bytes": 2 * t * d * (3 if case["residual"] else 1) + 2 * d + out, "flops": 6 * t * d}
    if op == "linear":
        t, k, n = case["T"], case["K"], case["N"]
        x = t * k + 4 * t * -(-k // GROUP) if case["fp8"] else 2 * t * k
        return {"bytes": x + n * k // 2 + 2 * n * -(-k // GROUP) + 2 * t * n, "flops": 2 * t * k * n}
    if op == "weights":
        n, k = case["N"], case["K"]
        return {"bytes": 2 * n * k + n * k // 2 + 2 * n * -(-k // GROUP) + 2 * n * k, "flops": 4 * n * k}
    tokens = max(1, sum(_lengths(case)))
    return {"bytes": tokens * (LATENT + 4 + 2 * ROPE + 2 * (LATENT + ROPE)), "flops": tokens * (LATENT + ROPE)}


def _to_8_bits(x):
    """E4M3 codes and a scale for each 128 columns, as a program that has 8-bit activations holds them."""
    t, d = x.shape
    g = -(-d // GROUP)
    p = torch.zeros(t, g * GROUP, device=x.device)
    p[:, :d] = x
    s = (p.view(t, g, GROUP).abs().amax(-1) / 448.0).clamp_min(FLOOR)
    q = (p.view(t, g, GROUP) / s[..., None]).clamp(-448.0, 448.0).view(t, -1)[:, :d]
    return q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, op = torch.device("cuda"), case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": dict(case)}
    if op == "norm":
        t, d = case["T"], case["D"]
        # a residual stream: a few columns far larger than the rest
        spread = torch.where(torch.rand(d, generator=g, device=dev) < 0.01, 20.0, 1.0)
        s["x"] = normal(t, d).to(torch.bfloat16)
        s["residual"] = s["residual_out"] = None
        if case["residual"]:
            s["residual"] = (normal(t, d) * spread).to(torch.bfloat16)
            s["residual_out"] = torch.empty_like(s["residual"])
        s["weight"] = (1.0 + 0.1 * normal(d)).to(torch.bfloat16)
    elif op == "linear":
        t, k, n = case["T"], case["K"], case["N"]
        low = (normal(n, k // 2) * 2.6).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        high = (normal(n, k // 2) * 2.6).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        s["w4"] = low | (high << 4)
        s["scale"] = ((0.5 + torch.rand(n, -(-k // GROUP), generator=g, device=dev)) / (2.6 * k ** 0.5)).to(torch.bfloat16)
        x = normal(t, k)
        if case["fp8"]:
            s["x"], s["x_scale"] = _to_8_bits(x)
        else:
            s["x"] = x.to(torch.bfloat16)
    elif op == "weights":
        s["w"] = (normal(case["N"], case["K"]) / case["K"] ** 0.5).to(torch.bfloat16)
    else:
        lens = _lengths(case)
        need = [-(-n // PAGE) for n in lens]
        pool = sum(need) + -(-sum(need) // 10) + 1
        perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        most = max(max(need), 1)
        slot = torch.arange(most, device=dev)
        counts = torch.tensor(need, device=dev)
        first = torch.cumsum(counts, 0) - counts
        place = (first[:, None] + slot).clamp_max(pool - 1)
        s["page_table"] = torch.where(slot < counts[:, None], perm[place], -1).to(torch.int32).contiguous()
        s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["max_kv_len"] = max(max(lens), 1)
        c = normal(pool * PAGE, LATENT)
        scale = (c.abs().amax(-1) / 448.0).clamp_min(2.0 ** -10)
        s["codes"] = (c / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(pool, PAGE, LATENT)
        s["scale"] = scale.view(pool, PAGE)
        s["keys"] = (normal(pool * PAGE, ROPE) / scale[:, None]).to(torch.float16).view(pool, PAGE, ROPE)
        s["rows"] = torch.zeros(len(lens) * most, PAGE, LATENT + ROPE, dtype=torch.bfloat16, device=dev)
    return s


def _groups(d, device):
    return torch.arange(d, device=device) // GROUP


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {} if s["residual"] is None else {"residual": h.to(torch.bfloat16)}
    if not s["case"]["fp8"]:
        return {**out, "y": y.to(torch.bfloat16)}
    t, d = y.shape
    a = torch.nn.functional.pad(y.abs(), (0, -d % GROUP)).view(t, -1, GROUP).amax(-1)
    scale = (a / 448.0).clamp_min(FLOOR)
    q = (y / scale[:, _groups(d, y.device)]).clamp(-448.0, 448.0)
    return {**out, "y8": q.to(torch.float8_e4m3fn), "scale": scale}


def _plain_weights(w4, scale):
    n, half = w4.shape
    c = torch.stack((w4 & 15, w4 >> 4), -1).view(n, 2 * half).float() - 8.0
    return c * scale.float()[:, _groups(2 * half, w4.device)]


def _plain_linear(s):
    x = s["x"]
    if s["case"]["fp8"]:
        x = x.view(torch.float8_e4m3fn).float() * s["x_scale"][:, _groups(x.shape[1], x.device)]
    return (x.float() @ _plain_weights(s["w4"], s["scale"]).t()).to(torch.bfloat16)


def _plain_quantise(s):
    w = s["w"].float()
    n, k = w.shape
    a = torch.nn.functional.pad(w.abs(), (0, -k % GROUP)).view(n, -1, GROUP).amax(-1)
    scale = torch.where(a > 0, a / 7.0, 1.0).to(torch.bfloat16)
    c = (w / scale.float()[:, _groups(k, w.device)]).round().clamp(-8, 7)
    return {"scale": scale, "weights": (c * scale.float()[:, _groups(k, w.device)]).to(torch.bfloat16)}


def _plain_read(s):
    pt, lens = s["page_table"], s["kv_lens"]
    b, most = pt.shape
    pages = pt.clamp_min(0).long().view(-1)
    scale = s["scale"][pages][..., None]
    c = s["codes"].view(torch.float8_e4m3fn)[pages].float() * scale
    k = s["keys"][pages].float() * scale
    rows = torch.cat((c, k), -1).view(b, most * PAGE, LATENT + ROPE)
    there = torch.arange(most * PAGE, device=pt.device) < lens[:, None]
    rows = torch.where(there[..., None], rows, s["rows"].view_as(rows).float())
    return rows.to(torch.bfloat16).view(b * most, PAGE, LATENT + ROPE)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_linear, "weights": _plain_quantise, "read": _plain_read}[op](s)
    from mla_absorbed_decode_absorb_gb300 import ops
    if op == "norm":
        out = {} if s["residual"] is None else {"residual": s["residual_out"]}
        if case["fp8"]:
            y8, scale = ops.mla_rms_norm_fp8(s["x"], s["weight"], EPS, s["residual"], s["residual_out"])
            return {**out, "y8": y8.view(torch.float8_e4m3fn), "scale": scale}
        return {**out, "y": ops.mla_rms_norm(s["x"], s["weight"], EPS, s["residual"], s["residual_out"])}
    if op == "linear":
        if case["fp8"]:
            return ops.mla_linear_w4_fp8(s["x"], s["x_scale"], s["w4"], s["scale"])
        return ops.mla_linear_w4(s["x"], s["w4"], s["scale"])
    if op == "weights":
        w4, scale = ops.mla_quantize_w4(s["w"])
        return {"scale": scale, "weights": ops.mla_dequantize_w4(w4, scale)}
    return ops.mla_read_kv_fp8((s["codes"], s["scale"], s["keys"]), s["page_table"], s["kv_lens"], s["max_kv_len"],
                               s["rows"])


def _e4m3_values(device):
    """The 256 values of OCP E4M3: sign, 4 exponent bits (bias 7), 3 mantissa bits; S.1111.111 is NaN."""
    v = [0.0] * 256
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if c & 127 == 127 else -x if c & 128 else x
    return torch.tensor(v, dtype=torch.float64, device=device)


def _e4m3_nearest(x):
    """x (64 bits) rounded to the nearest E4M3 value, ties to even, saturating at 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    dev, op = torch.device("cuda"), case["op"]
    if op == "norm":
        h = s["x"].double()
        out = {}
        if case["residual"]:
            h += s["residual"].double()
            out["residual"] = h.clone()
        t, d = h.shape
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / d + EPS)
        y *= s["weight"].double()
        if not case["fp8"]:
            return {**out, "y": y}
        scales, values = [], []
        for k in range(0, d, GROUP):
            part = y[:, k:k + GROUP]
            scale = torch.maximum(part.abs().max(1).values / 448.0, torch.tensor(FLOOR, dtype=torch.float64, device=dev))
            scales.append(scale)
            values.append(_e4m3_nearest(part / scale[:, None]))
        return {**out, "y8": torch.cat(values, 1), "scale": torch.stack(scales, 1)}
    if op == "linear":
        t, k, n = case["T"], case["K"], case["N"]
        x = _e4m3_values(dev)[s["x"].long()] if case["fp8"] else s["x"].double()
        y = torch.zeros(t, n, dtype=torch.float64, device=dev)
        for j in range(0, k, GROUP):
            part = s["w4"][:, j // 2:(j + GROUP) // 2].long()
            c = torch.empty(n, 2 * part.shape[1], dtype=torch.float64, device=dev)
            c[:, 0::2], c[:, 1::2] = (part % 16 - 8).double(), (part // 16 - 8).double()
            a = x[:, j:j + GROUP]
            if case["fp8"]:
                a = a * s["x_scale"][:, j // GROUP, None].double()
            y += a @ (c * s["scale"][:, j // GROUP, None].double()).t()
        return y
    if op == "weights":
        w = s["w"].double()
        scales, values = [], []
        for j in range(0, case["K"], GROUP):
            part = w[:, j:j + GROUP]
            top = part.abs().max(1).values
            scale = torch.where(top == 0, torch.ones_like(top), top / 7.0).to(torch.bfloat16).double()
            scales.append(scale)
            values.append(torch.clamp(torch.round(part / scale[:, None]), -8, 7) * scale[:, None])
        return {"scale": torch.stack(scales, 1), "weights": torch.cat(values, 1)}
    pt, lens = s["page_table"].cpu(), s["kv_lens"].cpu()
    rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=dev)
    table, most = _e4m3_values(dev), pt.shape[1]
    for b in range(pt.shape[0]):
        n = int(lens[b])
        if n == 0:
            continue
        pages = pt[b, :-(-n // PAGE)].long().to(dev)
        scale = s["scale"][pages].double().view(-1, 1)[:n]
        part = rows[b * most:(b + 1) * most].view(-1, LATENT + ROPE)
        part[:n, :LATENT] = table[s["codes"][pages].view(-1, LATENT)[:n].long()] * scale
        part[:n, LATENT:] = s["keys"][pages].view(-1, ROPE)[:n].double() * scale
    return rows
