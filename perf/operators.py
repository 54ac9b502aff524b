"""Cases of the 4-bit projections and of the state-pool operators: what each takes, computes
and returns, in a plain form and through the package.

Operators:
  quantize   bf16 rows -> microscaled 4-bit codes (E2M1) with a scale per block of a row, and back
             (the values that the codes stand for).  "nvfp4": blocks of 16, E4M3 block scales and a
             power of two per row; "mxfp4": blocks of 32, power-of-two block scales.
  project    in_proj / out_proj of the mixer on 4-bit operands: the hidden states are quantised row
             by row and multiplied with weights held in 4 bits; f32 sums, bf16 results.
  copy       pool rows (state and conv history) copied or forked by (source, destination) pairs, all
             reads before all writes, in place.
  compact    the pool's live rows moved to its front, freed rows cleared where asked for.

own = False computes the plain form with elementary torch operations, own = True calls the package.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32}
D, W1 = 128, 3  # head width, rows of a conv history


def listed():
    return [
        # hidden states of a 64-row decode batch, ahead of a product
        {"name": "quantize_decode64", "op": "quantize", "rows": 64, "k": 5120, "format": "nvfp4", "std": 1.0},
        # the stacked in_proj weights of one layer, quantised at load
        {"name": "quantize_weights_mx", "op": "quantize", "rows": 16480, "k": 5120, "format": "mxfp4", "std": 0.014},
        # one token of one row: latency, the weights read once
        {"name": "in_proj_decode1", "op": "project", "which": "in", "t": 1, "hidden": 5120, "kh": 16, "vh": 48,
         "format": "nvfp4"},
        # a decode batch of 64 rows
        {"name": "in_proj_decode64", "op": "project", "which": "in", "t": 64, "hidden": 5120, "kh": 16, "vh": 48,
         "format": "nvfp4"},
        # a small decode batch through the output projection
        {"name": "out_proj_decode8_mx", "op": "project", "which": "out", "t": 8, "hidden": 5120, "kh": 16, "vh": 48,
         "format": "mxfp4"},
        # an odd prompt through a small mixer: ragged tiles everywhere
        {"name": "in_proj_ragged_mx", "op": "project", "which": "in", "t": 333, "hidden": 1088, "kh": 4, "vh": 12,
         "format": "mxfp4"},
        # prefill of one row of 8192 tokens
        {"name": "in_proj_prefill8192", "op": "project", "which": "in", "t": 8192, "hidden": 5120, "kh": 16, "vh": 48,
         "format": "nvfp4"},
        # an odd prefill through the output projection
        {"name": "out_proj_prefill2049", "op": "project", "which": "out", "t": 2049, "hidden": 5120, "kh": 16,
         "vh": 48, "format": "nvfp4"},
        # one prompt's state forked to 4 continuations
        {"name": "copy_fork1to4", "op": "copy", "pool": 16, "kh": 16, "vh": 48, "forks": 1, "ways": 4, "reorder": 0,
         "width": 1},
        # 16 requests of 8 beams each reordered in place: parents drawn with repetition, so rows are
        # read, kept and overwritten within a request
        {"name": "copy_beams128", "op": "copy", "pool": 160, "kh": 16, "vh": 48, "forks": 0, "ways": 1, "reorder": 16,
         "width": 8},
        # a pool of 16 rows with a few ended sequences
        {"name": "compact16", "op": "compact", "pool": 16, "kh": 16, "vh": 48, "live": 0.7, "clear": True},
        # a server's pool half empty
        {"name": "compact192", "op": "compact", "pool": 192, "kh": 16, "vh": 48, "live": 0.5, "clear": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "project", "project", "copy", "compact"])
    heads = rng.choice([(16, 48), (16, 32), (8, 16), (4, 12), (2, 16), (3, 9)])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 16384), "k": 64 * _log(rng, 1, 80), "format": rng.choice(list(BLOCK)),
                "std": rng.choice([1.0, 0.014])}
    if op == "project":
        return {"op": op, "which": rng.choice(["in", "out"]), "t": _log(rng, 1, 8192), "hidden": 64 * _log(rng, 4, 80),
                "kh": heads[0], "vh": heads[1], "format": rng.choice(list(BLOCK))}
    if op == "copy":
        case = {"op": op, "pool": 0, "kh": heads[0], "vh": heads[1], "forks": rng.randint(0, 4),
                "ways": rng.randint(1, 8), "reorder": rng.randint(1, 12), "width": rng.randint(2, 9)}
        case["pool"] = case["forks"] * (1 + case["ways"]) + case["reorder"] * case["width"] + rng.randint(0, 7)
        return case
    return {"op": op, "pool": _log(rng, 4, 160), "kh": heads[0], "vh": heads[1],
            "live": rng.choice([0.2, 0.4, 0.6, 0.8]), "clear": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _widths(case):
    """(output widths, contraction width) of a projection; the stacked in_proj rows are qkv, z, b, a."""
    conv, value = (2 * case["kh"] + case["vh"]) * D, case["vh"] * D
    if case["which"] == "in":
        return [conv, value, case["vh"], case["vh"]], case["hidden"]
    return [case["hidden"]], value


def _pairs(case, gen):
    """(source, destination) rows of a copy: forks of one row to several, then reorderings of a
    request's rows by parents drawn with repetition."""
    rows = torch.randperm(case["pool"], generator=gen).tolist()
    src, dst = [], []
    for _ in range(case["forks"]):
        first = rows.pop()
        for _ in range(case["ways"]):
            src.append(first)
            dst.append(rows.pop())
    for _ in range(case["reorder"]):
        mine = [rows.pop() for _ in range(case["width"])]
        parents = torch.randint(case["width"], (case["width"],), generator=gen).tolist()
        src += [mine[p] for p in parents]
        dst += mine
    return src, dst


def _values(case, seed):
    """The inputs, from the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(shape, std):
        return torch.randn(shape, generator=gen, device=DEV) * std

    if case["op"] == "quantize":
        x = normal((case["rows"], case["k"]), case["std"])
        loud = torch.randint(case["k"], (1 + case["k"] // 256,), generator=host).to(DEV)  # a few loud channels
        x[:, loud] *= 12.0
        return {"x": x.to(torch.bfloat16)}
    if case["op"] == "project":
        outs, k = _widths(case)
        x = normal((case["t"], k), 1.0)
        loud = torch.randint(k, (1 + k // 256,), generator=host).to(DEV)
        x[:, loud] *= 12.0
        return {"x": x.to(torch.bfloat16), "w": normal((sum(outs), k), k ** -0.5).to(torch.bfloat16)}
    conv = (2 * case["kh"] + case["vh"]) * D
    state = {"state": normal((case["pool"], case["vh"], D, D), 0.05), "conv": normal((case["pool"], W1, conv), 1.0)}
    if case["op"] == "copy":
        state["src"], state["dst"] = _pairs(case, host)
    else:
        state["live"] = (torch.rand(case["pool"], generator=host) < case["live"]).tolist()
    return state


def prepare(case, seed):
    state = {"case": case, **_values(case, seed)}
    if case["op"] == "project":  # the weights are kept in 4 bits, laid out once
        w = state.pop("w")
        state["plain_w"] = _quantize(w, case["format"])
        if own:
            state["own_w"] = _package().quantize(w, case["format"])
    return state


def _package():
    import gated_deltanet_mixer_gdn_b200 as gdn
    return gdn


def _dims(case):
    return _package().Dims(num_k_heads=case["kh"], num_v_heads=case["vh"])


# ------------------------------------------------------------------ the plain form
def _power(e):
    """2^e in f32 from its bits, e in [-127, 127] (2^-127 is subnormal)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantize(x, fmt):
    """(2 * E2M1 value as int8 [rows, K], block scale f32 [rows, K / block], row scale f32 [rows, 1])."""
    rows, k = x.shape
    blocks = x.float().view(rows, k // BLOCK[fmt], BLOCK[fmt])
    top = blocks.abs().amax(2)
    if fmt == "nvfp4":
        # the smallest power of two that keeps every block scale within E4M3: amax <= 448 * 6 * row
        m, e = torch.frexp(top.amax(1, keepdim=True))  # m in [0.5, 1), 448 * 6 = 0.65625 * 2^12
        row = _power((e - 12 + (m > 0.65625).int()).clamp(min=-100))
        v = top / row / 6.0
        ve = (torch.frexp(v)[1] - 1).clamp(min=-6)  # E4M3: 3 fraction bits, normal down to 2^-6
        scale = torch.round(v / _power(ve - 3)) * _power(ve - 3)
    else:
        row = torch.ones((rows, 1), device=x.device)
        e = torch.frexp(top)[1] - 1 - 2  # floor(log2(amax)) - 2: the largest E2M1 value is 6 = 1.5 * 2^2
        scale = _power(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127))
    q = blocks / row.unsqueeze(2) / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(2)
    q = torch.where(scale.unsqueeze(2) > 0, q, torch.zeros_like(q))
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))  # E2M1: 0 .5 1 1.5 2 3 4 6, ties to even
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return (2 * torch.copysign(a, q)).to(torch.int8).view(rows, k), scale, row


def _dequantize(q):
    code, scale, row = q
    rows, k = code.shape
    v = (code.float() * 0.5).view(rows, scale.shape[1], -1) * scale.unsqueeze(2) * row.unsqueeze(2)
    return v.view(rows, k)


def _moves(live):
    """Live rows behind the live count fill the free rows before it, in ascending order."""
    n = sum(live)
    holes = [i for i in range(n) if not live[i]]
    movers = [i for i in range(n, len(live)) if live[i]]
    remap = [-1] * len(live)
    for i in range(len(live)):
        if live[i]:
            remap[i] = i
    for s, h in zip(movers, holes):
        remap[s] = h
    return movers, holes, remap, n


def _run_plain(state):
    case = state["case"]
    if case["op"] == "quantize":
        return _dequantize(_quantize(state["x"], case["format"])).to(torch.bfloat16)
    if case["op"] == "project":
        x = _dequantize(_quantize(state["x"], case["format"]))
        y = torch.matmul(x, _dequantize(state["plain_w"]).t()).to(torch.bfloat16)
        return [p.contiguous() for p in y.split(_widths(case)[0], 1)]
    if case["op"] == "copy":
        src = torch.tensor(state["src"], device=DEV)
        dst = torch.tensor(state["dst"], device=DEV)
        for pool in (state["state"], state["conv"]):
            pool.index_copy_(0, dst, pool.index_select(0, src))
        return [state["state"], state["conv"]]
    movers, holes, remap, n = _moves(state["live"])
    for pool in (state["state"], state["conv"]):
        if movers:
            src = torch.tensor(movers, device=DEV)
            dst = torch.tensor(holes, device=DEV)
            pool.index_copy_(0, dst, pool.index_select(0, src))
        if case["clear"]:
            pool[n:] = 0
    return [state["state"], state["conv"], torch.tensor(remap, dtype=torch.int32)]


# ------------------------------------------------------------------ through the package
def _run_own(state):
    gdn, case = _package(), state["case"]
    if case["op"] == "quantize":
        return gdn.dequantize(gdn.quantize(state["x"], case["format"]))
    if case["op"] == "project":
        if case["which"] == "in":
            qkv, z, a, b = gdn.in_proj_quant(state["x"], state["own_w"], dims=_dims(case))
            return [qkv, z, b, a]
        return [gdn.out_proj_quant(state["x"], state["own_w"], dims=_dims(case))]
    if case["op"] == "copy":
        gdn.copy_slots(state["src"], state["dst"], state["state"], state["conv"], dims=_dims(case))
        return [state["state"], state["conv"]]
    remap = gdn.compact_slots(state["live"], state["state"], state["conv"], clear=case["clear"], dims=_dims(case))
    return [state["state"], state["conv"], remap]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ sizes and the definition in 64 bits
def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["k"]
        held = n // 2 + n // BLOCK[case["format"]] + 4 * case["rows"]  # codes, block scales, row scales
        return {"bytes": 2 * n + 2 * held + 2 * n, "flops": 0}
    if case["op"] == "project":
        outs, k = _widths(case)
        n, t = sum(outs), case["t"]
        held = n * k // 2 + n * k // BLOCK[case["format"]] + 4 * n
        return {"bytes": 2 * t * k + held + 2 * t * n, "flops": 2 * t * n * k}
    row = 4 * (case["vh"] * D * D + W1 * (2 * case["kh"] + case["vh"]) * D)
    if case["op"] == "copy":
        # a row that is its own parent stays where it is; of a request's w rows, with parents drawn
        # uniformly, w - 1 are expected to be written and w (1 - (1 - 1/w)^(w-1)) read by another
        w = case["width"]
        moved = case["reorder"] * ((w - 1) + w * (1 - (1 - 1 / w) ** (w - 1)))
        return {"bytes": int(row * (case["forks"] * (1 + case["ways"]) + moved)), "flops": 0}
    n = case["pool"] * case["live"]
    moved = n * (1 - case["live"])
    cleared = case["pool"] - n if case["clear"] else 0
    return {"bytes": int(row * (2 * moved + cleared)), "flops": 0}


def _definition(x, fmt):
    """The quantised values in 64 bits.  Of the values that a format holds the nearest is taken, of two
    equally near ones the one with the even code; a table of the format's values decides, so no
    rounding enters."""
    rows, k = x.shape

    def nearest(v, table):
        hi = torch.bucketize(v, table).clamp(max=len(table) - 1)  # table[hi - 1] < v <= table[hi]
        lo = (hi - 1).clamp(min=0)
        mid = (table[lo] + table[hi]) / 2
        up = (v > mid) | ((v == mid) & (hi % 2 == 0))
        return table[torch.where(up, hi, lo)]

    fours = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    blocks = x.double().view(rows, k // BLOCK[fmt], BLOCK[fmt])
    top = blocks.abs().amax(2)
    if fmt == "nvfp4":
        eights = [m / 8 * 2.0 ** -6 for m in range(8)]
        eights += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
        eights = torch.tensor(eights, dtype=torch.float64, device=x.device)
        powers = torch.tensor([2.0 ** e for e in range(-100, 121)], dtype=torch.float64, device=x.device)
        row = powers[torch.bucketize(top.amax(1) / 2688.0, powers)].view(rows, 1)  # least power >= amax / 2688
        # top / (6 row) against E4M3's midpoints, both sides times 6 so that they are exact
        scale = nearest(top / row, 6 * eights) / 6
    else:
        row = torch.ones((rows, 1), dtype=torch.float64, device=x.device)
        powers = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device=x.device)
        scale = powers[(torch.bucketize(top / 4.0, powers, right=True) - 1).clamp(min=0)]
    out = torch.empty_like(blocks)
    part = max(1, (1 << 24) // k)
    for r in range(0, rows, part):  # in parts, the tables' indexes take room
        s = scale[r:r + part].unsqueeze(2) * row[r:r + part].unsqueeze(2)
        q = torch.where(s > 0, blocks[r:r + part] / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))
        out[r:r + part] = torch.copysign(nearest(q.abs(), fours), q) * s
    return out.view(rows, k)


def exact(case, seed):
    v = _values(case, seed)
    if case["op"] == "quantize":
        return _definition(v["x"], case["format"])
    if case["op"] == "project":
        y = torch.matmul(_definition(v["x"], case["format"]), _definition(v["w"], case["format"]).t())
        return [p.contiguous() for p in y.split(_widths(case)[0], 1)]
    if case["op"] == "copy":
        out = []
        for pool in (v["state"], v["conv"]):
            new = pool.clone()
            for s, d in zip(v["src"], v["dst"]):
                new[d] = pool[s]
            out.append(new.double())
        return out
    movers, holes, remap, n = _moves(v["live"])
    out = []
    for pool in (v["state"], v["conv"]):
        new = pool.double()
        for s, h in zip(movers, holes):
            new[h] = pool[s].double()
        if case["clear"]:
            new[n:] = 0
        out.append(new)
    return out + [torch.tensor(remap, dtype=torch.int32)]
