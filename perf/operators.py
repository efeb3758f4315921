"""Measured operators: scored routing to experts, MXFP4 quantisation, MXFP4 linear layers, MXFP4 expert layers.

`run` takes what `prepare` gives and makes one pass through an operator: in the
plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where `own` is true, by the calls that a user makes of bit_moe_expert_gb300.

MXFP4: blocks of 32 consecutive values along K share a power-of-two scale 2^e
(an E8M0 byte e + 127); a value is an E2M1 code (sign, two exponent bits, one
mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), two codes a byte, the lower index in
the low nibble.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def _route(T, E, k, score, bias, groups, kept, rows, top=2):
    return {"op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups, "kept": kept,
            "group_top": top, "scale": 2.5 if score == "sigmoid" else 1.0, "block_rows": rows}


def _layer(T, d, I, I_shared, E, k, score, bias, groups, kept, rows):
    return dict(_route(T, E, k, score, bias, groups, kept, rows), op="layer", d=d, I=I, I_shared=I_shared)


def listed():
    def named(name, case):
        return dict(case, name=name)

    return [
        # one decoded token of a 256-expert layer with a sigmoid router, its balance bias and 8 groups: pure latency
        named("route_decode", _route(1, 256, 8, "sigmoid", True, 8, 4, 16)),
        # a ragged prompt, an expert count that is no power of two, softmax scores without groups
        named("route_odd", _route(777, 130, 6, "softmax", False, 1, 1, 64)),
        # a long prompt's routing in one call: bias and groups over 4096 tokens
        named("route_prompt", _route(4096, 256, 8, "sigmoid", True, 8, 4, 128)),
        # the activations of a 512-token prompt at d = 2048
        named("quantize_prompt", {"op": "quantize", "rows": 512, "K": 2048, "x": "bf16"}),
        # a checkpoint's fp32 matrix being converted (a stack of 16 experts' 2816 x 704 projections)
        named("quantize_weights", {"op": "quantize", "rows": 16 * 704, "K": 2816, "x": "fp32"}),
        # one token through a 2048 -> 2048 projection: the weight stream and the launches count
        named("linear_decode", {"op": "linear", "T": 1, "K": 2048, "N": 2048, "x": "bf16", "y": "bf16"}),
        # a ragged batch, odd output width, fp16 in and fp32 out
        named("linear_odd", {"op": "linear", "T": 333, "K": 2816, "N": 1001, "x": "fp16", "y": "fp32"}),
        # a large square product: the tensor cores' rate
        named("linear_large", {"op": "linear", "T": 8192, "K": 8192, "N": 8192, "x": "bf16", "y": "bf16"}),
        # the decode workload's layer (d 2048, 256 experts, top 8 and a shared one) for one token
        named("layer_decode", _layer(1, 2048, 512, 512, 256, 8, "sigmoid", True, 8, 4, 16)),
        # the canvas workload's layer: 256 positions, 128 experts, I = 704 (no multiple of 128), softmax
        named("layer_canvas", _layer(256, 2816, 704, 0, 128, 8, "softmax", False, 1, 1, 32)),
        # the 512-token prefill layer: every expert active, the weight stream counts
        named("layer_prefill", _layer(512, 2048, 512, 512, 256, 8, "sigmoid", True, 8, 4, 32)),
        # the 4096-token prompt in one call
        named("layer_prompt", _layer(4096, 2048, 512, 512, 256, 8, "sigmoid", True, 8, 4, 128)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_route(rng, T, E):
    """A router over about E experts: with or without groups (E is then made a multiple of the groups)."""
    score = rng.choice(["softmax", "sigmoid"])
    groups = rng.choice([1, 1, 2, 4, 8])
    E = max(groups * 4, E // groups * groups)
    kept = 1 if groups == 1 else rng.randint(max(1, groups // 4), groups)
    k = rng.randint(1, min(12, kept * (E // groups)))
    return T, E, k, score, rng.random() < 0.6, groups, kept


def draw(rng):
    op = rng.choice(["route", "quantize", "linear", "layer"])
    if op == "route":
        T, E, k, score, bias, groups, kept = _draw_route(rng, _log(rng, 1, 4096), _log(rng, 16, 512))
        return _route(T, E, k, score, bias, groups, kept, rng.choice([16, 32, 48, 64, 128]), rng.choice([1, 2]))
    if op == "quantize":
        return {"op": "quantize", "rows": _log(rng, 1, 7500), "K": 32 * _log(rng, 4, 128),
                "x": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "linear":
        return {"op": "linear", "T": _log(rng, 1, 6000), "K": 32 * _log(rng, 4, 160), "N": _log(rng, 64, 6000),
                "x": rng.choice(["bf16", "fp16", "fp32"]), "y": rng.choice(["bf16", "fp32"])}
    T, E, k, score, bias, groups, kept = _draw_route(rng, _log(rng, 1, 2000), _log(rng, 8, 160))
    I = 32 * rng.randint(4, 22)
    rows = 16 if T * k < 16 * E else rng.choice([32, 64, 96, 128])
    return _layer(T, 32 * rng.randint(8, 80), I, rng.choice([0, I, 512]), E, k, score, bias, groups, kept, rows)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _unsettled(logits, bias, c):
    """Rows whose selection hangs on less than 32-bit rounding: two neighbours in the order, or the last group kept and
    the next one, closer than a few units in the last place of what they are sums of.  Such an order has no value in
    32 bits."""
    s = _scores(logits.double(), c)
    b = torch.zeros(c["E"], dtype=torch.float64, device="cuda") if bias is None else bias.double()
    choice = s + b
    unit = 4e-6 * (s + b.abs()).amax(1)
    bad = torch.zeros(logits.shape[0], dtype=torch.bool, device="cuda")
    if c["groups"] > 1:
        g = choice.view(logits.shape[0], c["groups"], -1).sort(dim=-1, descending=True)[0][..., :c["group_top"]].sum(-1)
        g, order = g.sort(dim=1, descending=True, stable=True)
        if c["kept"] < c["groups"]:
            bad |= g[:, c["kept"] - 1] - g[:, c["kept"]] < 2 * unit
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, order[:, :c["kept"]], True)
        choice = choice.masked_fill(~keep.repeat_interleave(c["E"] // c["groups"], 1), -math.inf)
    v = choice.sort(dim=1, descending=True)[0][:, :c["k"] + 1]
    return bad | (v[:, :-1] - v[:, 1:] < unit[:, None]).any(1)


def _logits(g, c):
    """Router logits N(0, 1) plus a fixed popularity of each expert, and the balance bias that works against it."""
    T, E = c["T"], c["E"]
    popular = 0.3 * _normal(g, E)
    logits = _normal(g, T, E) + popular
    scale = 0.1 if c["score"] == "sigmoid" else 0.3 / E
    bias = (scale * (_normal(g, E) - 2 * popular)).contiguous() if c["bias"] else None
    for _ in range(6):
        bad = _unsettled(logits, bias, c)
        n = int(bad.sum())
        if n == 0:
            break
        logits[bad] = _normal(g, n, E) + popular
    return logits, bias


def _pack(scale):
    """E8M0 bytes [E][N][K/32] -> the library's layout [E][ceil(N/128)][ceil(K/128)][512] (128 rows x 4 blocks a piece:
    byte 16 (r % 32) + 4 (r / 32) + block), rows and blocks past the end zero."""
    E, N, G = scale.shape
    n, g = -(-N // 128), -(-G // 4)
    p = torch.zeros((E, n * 128, g * 4), dtype=torch.uint8, device="cuda")
    p[:, :N, :G] = scale
    return p.view(E, n, 4, 32, g, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(E, n, g, 512)


def _encode(x):
    """fp32 [..., K] -> codes uint8 [..., K/2] and E8M0 bytes [..., K/32] (a checkpoint's matrix)."""
    v, e = _block_quantise(x)
    grid = torch.tensor(_GRID[1:], device="cuda")
    code = torch.bucketize(v.abs(), grid, right=True).to(torch.uint8) + ((v < 0).to(torch.uint8) << 3)
    code = code.view(*x.shape[:-1], x.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8).view(*x.shape[:-1], -1)


def _matrix(g, E, N, K):
    q, s = _encode(_normal(g, E, N, K) / math.sqrt(K))
    return {"q": q, "s": s, "sp": _pack(s)}


def _experts(g, E, d, I):
    return {"gate": _matrix(g, E, I, d), "up": _matrix(g, E, I, d), "down": _matrix(g, E, d, I)}


def _routing(c):
    """The caller's arrays that a routing writes."""
    T, E, k, rows = c["T"], c["E"], c["k"], c["block_rows"]
    i = dict(dtype=torch.int32, device="cuda")
    A = T * k
    return {"ids": torch.zeros((T, k), **i), "w": torch.zeros((T, k), dtype=torch.float32, device="cuda"),
            "counts": torch.zeros(E, **i), "offsets": torch.zeros(E + 1, **i), "perm": torch.zeros(A, **i),
            "inv_perm": torch.zeros(A, **i), "block_map": torch.zeros((-(-A // rows) + E, 3), **i),
            "num_blocks": torch.zeros(1, **i)}


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op in ("route", "layer"):
        st["logits"], st["bias"] = _logits(g, case)
        st["routing"] = _routing(case)
    if op == "quantize":
        # channels of different sizes, as activations and weights have
        rows, K = case["rows"], case["K"]
        st["x"] = (_normal(g, rows, K) * torch.exp(0.5 * _normal(g, K))).to(TYPES[case["x"]])
        st["values"] = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    if op == "linear":
        st["x"] = (_normal(g, case["T"], case["K"])).to(TYPES[case["x"]])
        st["weight"] = _matrix(g, 1, case["N"], case["K"])
        st["y"] = torch.empty((case["T"], case["N"]), dtype=TYPES[case["y"]], device="cuda")
    if op == "layer":
        st["x"] = _normal(g, case["T"], case["d"]).to(torch.bfloat16)
        st["routed"] = _experts(g, case["E"], case["d"], case["I"])
        st["shared"] = _experts(g, 1, case["d"], case["I_shared"]) if case["I_shared"] else None
        st["y"] = torch.empty((case["T"], case["d"]), dtype=torch.bfloat16, device="cuda")
        # the plain form's rows per expert: the largest count of this routing
        ids = _select(_scores(st["logits"], case), st["logits"], st["bias"], case)
        st["capacity"] = int(torch.bincount(ids.reshape(-1), minlength=case["E"]).max())
    return st


# ------------------------------------------------------------------ the plain form
def _scores(l, c):
    return l.softmax(1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-l))


def _select(s, l, bias, c):
    """The k experts of each row, the lower index first among equals."""
    choice = l if bias is None else s + bias
    if c["groups"] > 1:
        by = (s if bias is None else choice).view(l.shape[0], c["groups"], -1)
        g = by.sort(dim=-1, descending=True)[0][..., :c["group_top"]].sum(-1)
        order = g.sort(dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, order, True)
        choice = choice.masked_fill(~keep.repeat_interleave(c["E"] // c["groups"], 1), -math.inf)
    return choice.sort(dim=1, descending=True, stable=True)[1][:, :c["k"]]


def _plain_route(l, bias, c):
    T, E, k, rows = c["T"], c["E"], c["k"], c["block_rows"]
    s = _scores(l, c)
    ids = _select(s, l, bias, c)
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * c["scale"]
    flat = ids.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    ends = counts.cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    perm = flat.sort(stable=True)[1]
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device="cuda"))
    tiles = (counts + rows - 1) // rows
    tile_end = tiles.cumsum(0)
    b = torch.arange(-(-T * k // rows) + E, device="cuda")
    e = torch.searchsorted(tile_end, b, right=True).clamp(max=E - 1)
    at = (b - (tile_end - tiles)[e]) * rows
    block_map = torch.stack([e, offsets[e] + at, torch.minimum(counts[e] - at, torch.full_like(at, rows))], 1)
    block_map = torch.where((b < tile_end[-1])[:, None], block_map, 0)
    out = {"ids": ids, "counts": counts, "offsets": offsets, "perm": perm, "inv_perm": inv, "block_map": block_map,
           "num_blocks": tile_end[-1:]}
    out = {n: v.to(torch.int32) for n, v in out.items()}
    out["w"] = w.to(torch.float32) if l.dtype == torch.float32 else w
    return out


def _block_quantise(x):
    """E2M1 values (signed, in steps of the block's scale) [..., K/32, 32] and the scales' exponents [..., K/32, 1]."""
    b = x.view(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a)[1] - 3, -127).clamp(-127, 127)  # floor(log2 a) - 2
    v = torch.ldexp(b, -e).clamp(-6, 6)
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).to(v.dtype)
    return torch.round(v / step) * step, e


def _quantised(x):
    """x after a round trip through MXFP4."""
    v, e = _block_quantise(x)
    return torch.ldexp(v, e).view(x.shape)


def _decode(q):
    """The codes' E2M1 values [..., K]."""
    code = torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], -1)
    m = (code & 7).float()
    m = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(code >= 8, -m, m)


def _values(m):
    v = _decode(m["q"])
    e = m["s"].to(torch.int32)[..., None] - 127
    return torch.ldexp(v.view(*v.shape[:-1], -1, BLOCK), e).view(v.shape)


def _ffn(x, ex):
    """x [E][C][d] fp32 (MXFP4 values) through E experts."""
    gate = torch.matmul(x, _values(ex["gate"]).transpose(1, 2))
    up = torch.matmul(x, _values(ex["up"]).transpose(1, 2))
    h = _quantised(gate / (1 + torch.exp(-gate)) * up)
    return torch.matmul(h, _values(ex["down"]).transpose(1, 2))


def _rows_of(r, c, capacity):
    """Row c of expert e holds the assignment perm[offsets[e] + c]: the token of each, and each assignment's row."""
    A = c["T"] * c["k"]
    first = r["offsets"][:-1].long()
    at = torch.arange(capacity, device="cuda")[None, :]
    p = (first[:, None] + at).clamp(max=A - 1)
    token = torch.where(at < r["counts"][:, None], r["perm"].long()[p] // c["k"], 0)
    e = r["ids"].long().reshape(-1)
    return token, e * capacity + r["inv_perm"].long() - first[e]


def _plain_layer(st):
    c = st["case"]
    r = _plain_route(st["logits"], st["bias"], c)
    x = _quantised(st["x"].float())
    if 2 * c["T"] * c["k"] <= c["E"]:  # few assignments: the weights of each one's expert
        e = r["ids"].long().reshape(-1)
        taken = {n: {"q": m["q"][e], "s": m["s"][e]} for n, m in st["routed"].items()}
        y = _ffn(x.repeat_interleave(c["k"], 0)[:, None], taken).view(c["T"], c["k"], c["d"])
    else:
        token, row = _rows_of(r, c, st["capacity"])
        y = _ffn(x[token], st["routed"]).view(-1, c["d"])[row].view(c["T"], c["k"], c["d"])
    y = (y * r["w"][:, :, None]).sum(1)
    if st["shared"] is not None:
        y = y + _ffn(x[None], st["shared"])[0]
    return {"ids": r["ids"], "w": r["w"], "y": y.to(torch.bfloat16)}


def _plain(st):
    c = st["case"]
    if c["op"] == "route":
        return _plain_route(st["logits"], st["bias"], c)
    if c["op"] == "quantize":
        return _quantised(st["x"].float()).to(torch.bfloat16)
    if c["op"] == "linear":
        y = torch.matmul(_quantised(st["x"].float()), _values(st["weight"])[0].t())
        return y.to(TYPES[c["y"]])
    return _plain_layer(st)


# ------------------------------------------------------------------ the library's calls
def _handles(st):
    """The objects that a program keeps beside its tensors: they hold pointers to them and workspaces."""
    import bit_moe_expert_gb300 as bm
    c = st["case"]
    h = {"bm": bm}
    if c["op"] in ("route", "layer"):
        h["scoring"] = bm.Scoring(score=c["score"], bias=st["bias"], n_group=c["groups"], topk_group=c["kept"],
                                  group_top=c["group_top"], renormalize=True, scale=c["scale"])
        h["routing"] = bm.Routing(**st["routing"], block_rows=c["block_rows"])
    if c["op"] == "route":
        h["ws"] = bm.workspace(bm.moe_route_workspace_bytes(c["T"], c["E"], c["k"]))
    elif c["op"] == "quantize":
        h["m"] = bm.MxMat.empty(1, c["rows"], c["K"])
    elif c["op"] == "linear":
        h["w"] = bm.MxMat(st["weight"]["q"], st["weight"]["sp"])
        h["ws"] = bm.workspace(bm.moe_mx_linear_workspace_bytes(c["T"], c["N"], c["K"]))
    else:
        def experts(ex):
            return bm.MxExperts(**{n: bm.MxMat(m["q"], m["sp"]) for n, m in ex.items()})

        h["routed"] = experts(st["routed"])
        h["shared"] = experts(st["shared"]) if st["shared"] is not None else None
        h["ws"] = bm.workspace(bm.moe_mx_layer_workspace_bytes(c["T"], c["d"], c["I"], c["E"], c["k"], c["I_shared"],
                                                               c["block_rows"]))
    return h


def _kernels(st):
    c = st["case"]
    if "handles" not in st:
        st["handles"] = _handles(st)
    h = st["handles"]
    bm = h["bm"]
    if c["op"] == "route":
        bm.moe_route_scored(st["logits"], h["scoring"], c["k"], c["block_rows"], h["routing"], h["ws"])
        return st["routing"]
    if c["op"] == "quantize":
        bm.moe_mx_quantize(st["x"], h["m"])
        bm.moe_mx_dequant(h["m"], st["values"])
        return st["values"]
    if c["op"] == "linear":
        bm.moe_mx_linear(st["x"], h["w"], st["y"], h["ws"])
        return st["y"]
    bm.moe_mx_layer(st["logits"], h["scoring"], st["x"], h["routed"], h["shared"], c["k"], c["block_rows"],
                    h["routing"], st["y"], h["ws"])
    return {"ids": st["routing"]["ids"], "w": st["routing"]["w"], "y": st["y"]}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _mx_bytes(n):
    return n / 2 + n / BLOCK


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * (BYTES[c["x"]] + 2), "flops": 3 * n}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": T * K * BYTES[c["x"]] + _mx_bytes(N * K) + T * N * BYTES[c["y"]], "flops": 2 * T * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    route = T * E * 4 + T * k * 16 + 8 * E + 12 * min(T * k, T * k / c["block_rows"] + E)
    if c["op"] == "route":
        return {"bytes": route, "flops": 8 * T * E}
    active = E * (1 - (1 - k / E) ** T)  # experts that some token takes, at about even popularity
    weights = _mx_bytes(3 * c["d"] * (active * c["I"] + c["I_shared"]))
    return {"bytes": route + weights + 4 * T * c["d"], "flops": 6 * T * c["d"] * (k * c["I"] + c["I_shared"])}


# ------------------------------------------------------------------ in 64 bits
# MXFP4 operands are small multiples of one half times powers of two: the
# product over one block of 32 is exact in 32 bits (below 2^14 in units of 1/4),
# so blocks are multiplied in 32 bits, scaled and added up in 64.
_GRID = (0, .5, 1, 1.5, 2, 3, 4, 6)


def _exact_codes(x):
    """fp64 [..., K]: E2M1 values (fp32) and scales 2^e (fp64) by the nearest value of the grid, ties to the even code."""
    b = x.unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1)
    e = torch.where(a > 0, torch.floor(torch.log2(a)), torch.full_like(a, -125))
    e = e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a).double() * (a > 0)  # log2's own rounding
    scale = torch.exp2((e - 2).clamp(-127, 127))
    m = (b.abs() / scale[..., None]).clamp(max=6)
    v = torch.zeros_like(m)
    for i in range(7):  # past the midpoint of two neighbours, or on it where the upper one's code is even
        mid = (_GRID[i] + _GRID[i + 1]) / 2
        v = torch.where((m > mid) | ((m == mid) & (i % 2 == 1)), torch.full_like(m, _GRID[i + 1]), v)
    return (v * torch.sign(b)).flatten(-2).float(), scale


def _exact_weight(m):
    low, high = (m["q"] & 15).long(), (m["q"] >> 4).long()
    code = torch.stack([low, high], -1).flatten(-2)
    grid = torch.tensor(_GRID, device="cuda", dtype=torch.float32)
    return grid[code & 7] * (1 - 2 * (code >> 3)).float(), torch.exp2(m["s"].double() - 127)


def _exact_product(x, w):
    """[E][C][K] times [E][N][K], transposed, for (values, scales) of each."""
    (xv, xs), (wv, ws) = x, w
    total = 0
    for b in range(xs.shape[-1]):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        part = torch.bmm(xv[..., at], wv[..., at].transpose(1, 2)).double()
        part *= xs[..., b, None]
        part *= ws[..., b][:, None, :]
        total = part if b == 0 else total.add_(part)
    return total


def _exact_ffn(x, ex):
    gate = _exact_product(x, _exact_weight(ex["gate"]))
    up = _exact_product(x, _exact_weight(ex["up"]))
    h = gate * torch.sigmoid(gate) * up
    return _exact_product(_exact_codes(h), _exact_weight(ex["down"]))


def _exact_route(l, bias, c):
    """Row by row from the definition, on the host."""
    import numpy as np
    l = l.double().cpu().numpy()
    T, E, k = c["T"], c["E"], c["k"]
    if c["score"] == "softmax":
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = 1 / (1 + np.exp(-l))
    choice = s if bias is None else s + bias.double().cpu().numpy()
    size = E // c["groups"]
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        best = [sum(sorted(choice[t, g * size:(g + 1) * size], reverse=True)[:c["group_top"]]) for g in range(c["groups"])]
        kept = sorted(range(c["groups"]), key=lambda g: (-best[g], g))[:c["kept"]]
        among = sorted((e for g in kept for e in range(g * size, (g + 1) * size)), key=lambda e: (-choice[t, e], e))
        ids[t] = among[:k]
        w[t] = s[t, ids[t]] / s[t, ids[t]].sum() * c["scale"]
    lists = [[] for _ in range(E)]
    for a, e in enumerate(ids.reshape(-1)):
        lists[e].append(a)
    perm = np.array([a for x in lists for a in x], np.int32)
    inv = np.zeros(T * k, np.int32)
    inv[perm] = np.arange(T * k, dtype=np.int32)
    counts = np.array([len(x) for x in lists], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = c["block_rows"]
    tiles = [(e, offsets[e] + i, min(rows, counts[e] - i)) for e in range(E) for i in range(0, counts[e], rows)]
    block_map = np.zeros((-(-T * k // rows) + E, 3), np.int32)
    block_map[:len(tiles)] = tiles
    return {"ids": ids, "w": w, "counts": counts, "offsets": offsets, "perm": perm, "inv_perm": inv,
            "block_map": block_map, "num_blocks": np.array([len(tiles)], np.int32)}


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "route":
        return _exact_route(st["logits"], st["bias"], c)
    if c["op"] == "quantize":
        v, s = _exact_codes(st["x"].double())
        return v.double() * s.repeat_interleave(BLOCK, -1)
    if c["op"] == "linear":
        return _exact_product([t[None] for t in _exact_codes(st["x"].double())], _exact_weight(st["weight"]))[0]
    r = {n: torch.from_numpy(v).cuda() for n, v in _exact_route(st["logits"], st["bias"], c).items()}
    token, row = _rows_of(r, c, st["capacity"])
    x = _exact_codes(st["x"].double())
    y = _exact_ffn([t[token] for t in x], st["routed"]).view(-1, c["d"])[row].view(c["T"], c["k"], c["d"])
    y = (y * r["w"][:, :, None]).sum(1)
    if st["shared"] is not None:
        y = y + _exact_ffn([t[None] for t in x], st["shared"])[0]
    return {"ids": r["ids"], "w": r["w"], "y": y}
