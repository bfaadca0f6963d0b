"""What is measured of the expert products, their weight gradients, the 8-bit
block quantization and the 8-bit block-scaled products.

Notation: rows (tokens) are sorted by group (expert) and `offsets` holds
groups + 1 ascending row numbers; group g owns rows offsets[g] .. offsets[g+1].

  grouped   D[i] = alpha * A[i] . B[g] + beta * C[i]        for the rows i of group g
  wgrad     D[g] = alpha * X_g^T . Y_g + beta * C[g]        X_g, Y_g: the rows of group g
  quant     s = max(amax(block), 2^-100) / 448 (e5m2: 57344),
            q = round8(x * (448 / max(amax(block), 2^-100)))
  scaled    D[i,j] = sum over k-blocks b of sA[i,b] * sB[j/128,b] * (A8[i,b] . B8[j,b])

The plain forms compute the same in 32 bits with one torch product per group
(per block of 128 where the scales differ) and round once at the end.
"""
import math
import random

import numpy as np
import torch

own = False

_F = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
_TOP = {"e4m3": 448.0, "e5m2": 57344.0}
_LEAST = 2.0 ** -100


def listed():
    return [
        # one decoding step of a small model: a token for each of four experts (launch latency)
        {"name": "grouped_token", "op": "grouped", "dtype": "f16", "out": "f16", "groups": 4, "rows": 4, "tail": 0,
         "k": 512, "n": 512, "b_col": True, "skew": 0.0, "beta": 0.0},
        # decoding with a batch of 64 tokens spread unevenly over 64 experts, some of which get
        # none (bound by reading the experts' weights)
        {"name": "grouped_decode", "op": "grouped", "dtype": "bf16", "out": "bf16", "groups": 64, "rows": 64, "tail": 0,
         "k": 4096, "n": 1024, "b_col": True, "skew": 0.7, "beta": 0.0},
        # a training or prompt step: 16384 tokens over 8 experts (bound by the matrix units)
        {"name": "grouped_prompt", "op": "grouped", "dtype": "bf16", "out": "bf16", "groups": 8, "rows": 16384, "tail": 0,
         "k": 4096, "n": 4096, "b_col": True, "skew": 0.3, "beta": 0.0},
        # the same product's input gradient over many experts, from the weights as they are stored
        # (row-major here), added to a gradient that is there; ragged sizes, rows behind the last
        # group (padding of the batch) that have to stay as they were
        {"name": "grouped_input_grad", "op": "grouped", "dtype": "f16", "out": "f32", "groups": 32, "rows": 5003, "tail": 37,
         "k": 2056, "n": 1000, "b_col": False, "skew": 0.5, "beta": 1.0},
        # weight gradients of the training step: sums over each expert's tokens
        {"name": "wgrad_step", "op": "wgrad", "dtype": "bf16", "out": "bf16", "groups": 8, "rows": 16384, "tail": 0,
         "k": 2048, "n": 4096, "skew": 0.3, "beta": 0.0},
        # small experts, some without tokens, accumulated in 32 bits over micro-batches
        {"name": "wgrad_accumulate", "op": "wgrad", "dtype": "f16", "out": "f32", "groups": 24, "rows": 3001, "tail": 11,
         "k": 520, "n": 1032, "skew": 1.2, "beta": 1.0},
        # activations of a prompt on their way into an 8-bit product
        {"name": "quant_rows", "op": "quant", "dtype": "bf16", "q": "e4m3", "batch": 1, "m": 8192, "k": 4096, "block": 1,
         "transposed": False},
        # the activation of one token (launch latency)
        {"name": "quant_token", "op": "quant", "dtype": "f16", "q": "e4m3", "batch": 1, "m": 1, "k": 4096, "block": 1,
         "transposed": False},
        # experts' weights, stored K x N, into the 8-bit form that the product reads (N rows of K)
        {"name": "quant_weights", "op": "quant", "dtype": "bf16", "q": "e4m3", "batch": 8, "m": 4096, "k": 2048, "block": 128,
         "transposed": True},
        # the dense 4096^3 product in 8 bits
        {"name": "scaled_square", "op": "scaled", "a": "e4m3", "b": "e4m3", "out": "bf16", "groups": 0, "rows": 4096,
         "tail": 0, "k": 4096, "n": 4096, "skew": 0.0},
        # decoding 16 sequences through one 8-bit layer (bound by reading the weights)
        {"name": "scaled_decode", "op": "scaled", "a": "e4m3", "b": "e4m3", "out": "bf16", "groups": 0, "rows": 16,
         "tail": 0, "k": 4096, "n": 8192, "skew": 0.0},
        # experts' input gradient in 8 bits: e5m2 gradients by e4m3 weights, ragged, with padding rows
        {"name": "scaled_experts", "op": "scaled", "a": "e5m2", "b": "e4m3", "out": "f32", "groups": 16, "rows": 8011,
         "tail": 21, "k": 2064, "n": 4096, "skew": 0.5},
    ]


def _spread(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "wgrad", "quant", "scaled", "scaled"])
    step = rng.choice([1, 8, 8, 8, 64, 128])  # most widths are whole granules, some are odd
    if op == "quant":
        block = rng.choice([1, 128])
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "q": rng.choice(["e4m3", "e5m2"]),
                "batch": rng.choice([1, 1, 3, 8]), "m": _spread(rng, 1, 4096), "k": _spread(rng, 64, 4096, step),
                "block": block, "transposed": rng.random() < 0.4}
    groups = _spread(rng, 1, 64)
    rows = _spread(rng, 1, 8192)
    k, n = _spread(rng, 64, 4096, step), _spread(rng, 64, 4096, step)
    tail, skew = rng.choice([0, 0, 5, 130]), rng.choice([0.0, 0.4, 1.5])
    beta = rng.choice([0.0, 0.0, 1.0, 0.5])
    dtype = rng.choice(["bf16", "f16"])
    if op == "grouped":
        return {"op": op, "dtype": dtype, "out": rng.choice([dtype, "f32"]), "groups": groups, "rows": rows, "tail": tail,
                "k": k, "n": n, "b_col": rng.random() < 0.5, "skew": skew, "beta": beta}
    while groups * k * n > 1 << (27 if op == "wgrad" else 28):  # no more weights than the largest listed case has
        groups //= 2
    if op == "wgrad":
        return {"op": op, "dtype": dtype, "out": rng.choice([dtype, "f32"]), "groups": groups, "rows": rows, "tail": tail,
                "k": k, "n": n, "skew": skew, "beta": beta}
    if rng.random() < 0.5:
        groups = tail = 0
    return {"op": op, "a": rng.choice(["e4m3", "e4m3", "e5m2"]), "b": rng.choice(["e4m3", "e4m3", "e5m2"]),
            "out": rng.choice(["bf16", "f16", "f32"]), "groups": groups, "rows": rows, "tail": tail, "k": k, "n": n,
            "skew": skew}


def _counts(case):
    """Rows of each group, largest first: shares that fall as 1 / (rank + 1)^skew."""
    w = np.arange(1, case["groups"] + 1, dtype=np.float64) ** -case["skew"]
    c = np.floor(case["rows"] * w / w.sum()).astype(np.int64)
    left = case["rows"] - int(c.sum())
    c[:left % len(c)] += 1
    c += left // len(c)
    return [int(x) for x in c]


def _offsets(case, seed):
    if not case["groups"]:
        return [0, case["rows"]]
    c = _counts(case)
    random.Random(seed).shuffle(c)
    return [0] + [int(x) for x in np.cumsum(c)]


def _blocks(n):
    return -(-n // 128)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)

    if case["op"] == "quant":
        b, m, k = case["batch"], case["m"], case["k"]
        # activations and weights with a spread of magnitudes from row to row
        x = normal(b, k, m).to(_F[case["dtype"]]).transpose(1, 2) if case["transposed"] else \
            (normal(b, m, k) * torch.exp(normal(b, m, 1))).to(_F[case["dtype"]])
        s["x"] = x if b > 1 else x[0]
        return s
    groups, total, k, n = case["groups"], case["rows"] + case["tail"], case["k"], case["n"]
    s["host_offsets"] = _offsets(case, seed)
    s["offsets"] = torch.tensor(s["host_offsets"], device="cuda", dtype=torch.int64)
    if case["op"] == "scaled":
        # 8-bit operands as the quantization leaves them: block maxima near the type's largest value
        # and scales from row to row over a few powers of two
        kp = -(-k // 16) * 16
        e = max(1, groups)

        def operand(lead, rows, t, block):
            x = normal(lead, rows, kp)
            x[:, :, k:] = 0
            q = (x * (_TOP[t] / 8.0)).clamp_(-_TOP[t], _TOP[t]).to(_F[t])
            sc = torch.exp2(normal(lead, _blocks(k), -(-rows // block))) * (1.0 / _TOP[t])
            return q, sc.transpose(1, 2)

        aq, asc = operand(1, total, case["a"], 1)
        bq, bsc = operand(e, n, case["b"], 128)
        s["a"], s["a_scale"] = aq[0], asc[0]
        s["b"], s["b_scale"] = (bq, bsc) if groups else (bq[0], bsc[0])
        s["out"] = normal(total, n, dtype=_F[case["out"]])
        return s
    dt = _F[case["dtype"]]
    if case["op"] == "grouped":
        s["A"] = normal(total, k, dtype=dt)
        sc = 1.0 / math.sqrt(k)
        s["B"] = torch.stack([normal(n, k, dtype=dt, scale=sc) for _ in range(groups)]).transpose(1, 2) if case["b_col"] else \
            torch.stack([normal(k, n, dtype=dt, scale=sc) for _ in range(groups)])
        s["C"] = normal(total, n, dtype=_F[case["out"]])
    else:
        s["X"] = normal(total, k, dtype=dt)
        s["Y"] = normal(total, n, dtype=dt, scale=0.1)
        s["C"] = normal(groups, k, n, dtype=_F[case["out"]])
    s["out"] = s["C"].clone()  # rows that no group owns keep what is here
    return s


def _dequant(q, scale, block, k, to):
    """The values that an 8-bit operand stands for: its bytes by their blocks' scales."""
    rows = q.shape[-2]
    sc = scale.to(to).repeat_interleave(128, dim=-1)[..., :k]
    if block > 1:
        sc = sc.repeat_interleave(block, dim=-2)[..., :rows, :]
    return q[..., :k].to(to) * sc


def _per_group(case, s, to):
    """The operators' results in type `to`, one product per group."""
    o, off = s["out"], s["host_offsets"]
    if case["op"] == "wgrad":
        d = case["beta"] * s["C"].to(to) if case["beta"] else torch.zeros(s["C"].shape, device="cuda", dtype=to)
        for i in range(case["groups"]):
            lo, hi = off[i], off[i + 1]
            if hi > lo:
                d[i] += s["X"][lo:hi].to(to).t().contiguous() @ s["Y"][lo:hi].to(to)
        return d
    d = o.to(to).clone()
    if case["op"] == "grouped":
        for i in range(case["groups"]):
            lo, hi = off[i], off[i + 1]
            if hi > lo:
                d[lo:hi] = s["A"][lo:hi].to(to) @ s["B"][i].to(to).contiguous()
                if case["beta"]:
                    d[lo:hi] += case["beta"] * s["C"][lo:hi].to(to)
        return d
    k = case["k"]
    for i in range(max(1, case["groups"])):
        lo, hi = off[i], off[i + 1]
        if hi > lo:
            b = (s["b"][i], s["b_scale"][i]) if case["groups"] else (s["b"], s["b_scale"])
            a8 = _dequant(s["a"][lo:hi], s["a_scale"][lo:hi], 1, k, to)
            d[lo:hi] = a8 @ _dequant(*b, 128, k, to).t().contiguous()
    return d


def _quant_plain(case, x, to):
    """(values before they are rounded to 8 bits, scales) of x, its blocks' largest magnitudes in type `to`."""
    top, block = _TOP[case["q"]], case["block"]
    x = x.to(to)
    m, k = x.shape[-2:]
    pm, pk = -(-m // block) * block, _blocks(k) * 128
    p = torch.nn.functional.pad(x, (0, pk - k, 0, pm - m))
    p = p.reshape(*x.shape[:-2], pm // block, block, pk // 128, 128)
    amax = p.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(_LEAST)
    v = (p * (top / amax)).reshape(*x.shape[:-2], pm, pk)[..., :m, :k]
    return v, (amax / top).squeeze(-1).squeeze(-2)


def run(s):
    case = s["case"]
    if own:
        import dense_mixed_precision_02_amd as dmp
        if case["op"] == "grouped":
            c = s["C"] if case["beta"] else None
            return dmp.gemm_grouped(s["A"], s["B"], s["offsets"], c, out=s["out"], beta=case["beta"])
        if case["op"] == "wgrad":
            c = s["C"] if case["beta"] else None
            return dmp.gemm_grouped_wgrad(s["X"], s["Y"], s["offsets"], c, out=s["out"], beta=case["beta"])
        if case["op"] == "quant":
            r = dmp.quant8(s["x"], block=case["block"], dtype=_F[case["q"]])
            return {"q": r.q[..., :case["k"]], "scale": r.scale}
        a8 = dmp.Scaled8(s["a"], s["a_scale"], block=1, K=case["k"])
        b8 = dmp.Scaled8(s["b"], s["b_scale"], block=128, K=case["k"])
        return dmp.gemm_scaled8(a8, b8, s["offsets"] if case["groups"] else None, out=s["out"])
    if case["op"] == "quant":
        v, scale = _quant_plain(case, s["x"], torch.float32)
        return {"q": v.to(_F[case["q"]]), "scale": scale}
    return _per_group(case, s, torch.float32).to(s["out"].dtype)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "quant":
        return _exact_products(case, s)
    top, x = _TOP[case["q"]], s["x"].double()
    lead, (m, k) = x.shape[:-2], x.shape[-2:]
    block = case["block"]
    scale = torch.empty(*lead, -(-m // block), _blocks(k), device="cuda", dtype=torch.float64)
    v = torch.empty_like(x)
    for b in range(_blocks(k)):
        part = x[..., 128 * b:128 * b + 128]
        row = part.abs().amax(-1)
        if block > 1:
            row = torch.nn.functional.pad(row, (0, scale.shape[-2] * block - m)).unflatten(-1, (-1, block)).amax(-1)
        row = row.clamp_min(_LEAST)
        scale[..., b] = row / top
        v[..., 128 * b:128 * b + 128] = part * (top / row.repeat_interleave(block, -1)[..., :m, None])
    # rounding to 8 bits from 64: to the nearest multiple of the value's last place, ties to even
    mant, low = (3, -6) if case["q"] == "e4m3" else (2, -14)
    place = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - mant)
    return {"q": torch.round(v / place) * place, "scale": scale}


def _exact_products(case, s):
    """Row by row of the definition in 64 bits: each row's product with its own group's matrix."""
    off = s["host_offsets"]
    f = torch.float64
    if case["op"] == "wgrad":
        c = case["beta"] * s["C"].to(f)
        return torch.stack([c[i] + torch.matmul(s["X"][a:b].to(f).t(), s["Y"][a:b].to(f))
                            for i, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    rows = []
    for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if case["op"] == "grouped":
            rows.append(torch.matmul(s["A"][a:b].to(f), s["B"][i].to(f)) + case["beta"] * s["C"][a:b].to(f))
            continue
        bq, bs = (s["b"][i], s["b_scale"][i]) if case["groups"] else (s["b"], s["b_scale"])
        acc = torch.zeros(b - a, case["n"], device="cuda", dtype=f)
        for kb in range(_blocks(case["k"])):
            lo, hi = 128 * kb, min(case["k"], 128 * kb + 128)
            p = torch.matmul(s["a"][a:b, lo:hi].to(f), bq[:, lo:hi].to(f).t())
            acc += p * s["a_scale"][a:b, kb].to(f)[:, None] * bs[:, kb].to(f).repeat_interleave(128)[:case["n"]]
        rows.append(acc)
    rows.append(s["out"][off[-1]:].to(f))
    return torch.cat(rows)


def work(case):
    if case["op"] == "quant":
        e = case["batch"] * case["m"] * case["k"]
        nb = case["batch"] * -(-case["m"] // case["block"]) * _blocks(case["k"])
        return {"bytes": e * (_SIZE[case["dtype"]] + 1) + 4 * nb, "flops": 2 * e}
    t, k, n, o = case["rows"], case["k"], case["n"], _SIZE[case["out"]]
    used = sum(c > 0 for c in _counts(case)) if case["groups"] else 1
    if case["op"] == "grouped":
        moved = 2 * (t * k + used * k * n) + o * t * n * (2 if case["beta"] else 1)
    elif case["op"] == "wgrad":
        moved = 2 * t * (k + n) + o * case["groups"] * k * n * (2 if case["beta"] else 1)
    else:
        moved = t * k + used * k * n + o * t * n + 4 * _blocks(k) * (t + used * _blocks(n))
    return {"bytes": moved, "flops": 2 * t * k * n}
