"""Measured operators: 8-bit floating point with block scales (quantisation, linear layers, expert layers) and the RMS
norm that feeds them.

`run` takes what `prepare` gives and makes one pass through an operator: in the
plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where `own` is true, by the calls that a user makes of bit_moe_expert_gb300.

The format: E4M3 codes (the values of torch.float8_e4m3fn, up to 448).  Weights
[E][N][K] have one fp32 scale per 128 x 128 block, [E][ceil(N/128)][ceil(K/128)];
activations [rows][K] one per 128 columns of a row, [ceil(K/128)][rows up to a
multiple of 4].  Quantisation makes scales that are powers of two: the least 2^e,
e >= -126, with max |block| <= 448 2^e.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "blk": 1 + 4 / BLOCK}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _norm(T, d, x, residual, y):
    """residual: the type of the residual stream, or "none"; y: an output of x's type beside the 8-bit one."""
    return {"op": "norm", "T": T, "d": d, "x": x, "residual": residual, "y": y}


def _linear(T, K, N, x, y):
    """x: the activations' type, "blk" for such that a norm has quantised already."""
    return {"op": "linear", "T": T, "K": K, "N": N, "x": x, "y": y}


def _layer(T, d, I, I_shared, E, k, rows, x):
    return {"op": "layer", "T": T, "d": d, "I": I, "I_shared": I_shared, "E": E, "k": k, "block_rows": rows, "x": x}


def listed():
    def named(name, case):
        return dict(case, name=name)

    return [
        # one decoded token between two layers: the residual's addition, the norm, bf16 for the router, 8 bits for the experts
        named("norm_decode", _norm(1, 2048, "bf16", "bf16", True)),
        # a ragged batch whose residual stream is kept in fp32, 22 blocks a row
        named("norm_odd", _norm(777, 2816, "bf16", "fp32", True)),
        # a long prompt's rows at the large product's width: memory alone counts
        named("norm_prompt", _norm(8192, 8192, "bf16", "bf16", False)),
        # the activations of a 512-token prompt at d = 2048
        named("quantize_prompt", {"op": "quantize", "kind": "rows", "E": 1, "N": 512, "K": 2048, "x": "bf16"}),
        # a checkpoint's fp32 matrices being converted: a stack of 16 experts' 704 x 2816 projections, half blocks at the end
        named("quantize_weights", {"op": "quantize", "kind": "weights", "E": 16, "N": 704, "K": 2816, "x": "fp32"}),
        # one token through a 2048 -> 2048 projection: the weight stream and the launches count
        named("linear_decode", _linear(1, 2048, 2048, "bf16", "bf16")),
        # a ragged batch, odd output width, fp16 in and fp32 out
        named("linear_odd", _linear(333, 2816, 1001, "fp16", "fp32")),
        # a large square product: the tensor cores' rate
        named("linear_large", _linear(8192, 8192, 8192, "bf16", "bf16")),
        # the decode workload's layer (d 2048, 256 experts, top 8 and a shared one) for one token
        named("layer_decode", _layer(1, 2048, 512, 512, 256, 8, 16, "bf16")),
        # the canvas workload's layer: 256 positions, 128 experts, I = 704 (no multiple of 128)
        named("layer_canvas", _layer(256, 2816, 704, 0, 128, 8, 32, "bf16")),
        # the 512-token prefill layer behind a norm: every expert active, the weight stream counts
        named("layer_prefill", _layer(512, 2048, 512, 512, 256, 8, 32, "blk")),
        # the 4096-token prompt in one call
        named("layer_prompt", _layer(4096, 2048, 512, 512, 256, 8, 128, "bf16")),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "layer", "layer"])
    if op == "norm":
        x = rng.choice(["bf16", "fp16", "fp32"])
        return _norm(_log(rng, 1, 8000), 16 * _log(rng, 8, 500), x, rng.choice(["none", x, "fp32"]), rng.random() < 0.6)
    if op == "quantize":
        return {"op": "quantize", "kind": rng.choice(["rows", "weights"]), "E": rng.choice([1, 1, 2, 5]),
                "N": _log(rng, 1, 3000), "K": 16 * _log(rng, 4, 256), "x": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "linear":
        return _linear(_log(rng, 1, 6000), 16 * _log(rng, 8, 320), _log(rng, 64, 6000),
                       rng.choice(["bf16", "fp16", "fp32", "blk"]), rng.choice(["bf16", "fp16", "fp32"]))
    T, E = _log(rng, 1, 2000), _log(rng, 8, 160)
    k = rng.randint(1, min(12, E))
    I = 32 * rng.randint(4, 22)
    rows = 16 if T * k < 16 * E else rng.choice([32, 64, 96, 128])
    return _layer(T, 32 * rng.randint(8, 80), I, rng.choice([0, I, 512]), E, k, rows, rng.choice(["bf16", "blk"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _blocks(n):
    return -(-n // BLOCK)


def _padded(x, rows=False):
    """Zeros behind the last column (and the last row) up to whole blocks."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % BLOCK, 0, -x.shape[-2] % BLOCK if rows else 0))


def _matrix(g, E, N, K):
    """A checkpoint's matrix: codes uint8 [E][N][K], and scales max / 448 of each block, no powers of two."""
    w = _normal(g, E, N, K) / math.sqrt(K)
    b = _padded(w, rows=True).view(E, _blocks(N), BLOCK, _blocks(K), BLOCK)
    s = b.abs().amax((2, 4)) / 448
    full = s.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[..., :K]
    return {"q": (w / full).clamp(-448, 448).to(E4M3).view(torch.uint8), "s": s}


def _experts(g, E, d, I):
    return {"gate": _matrix(g, E, I, d), "up": _matrix(g, E, I, d), "down": _matrix(g, E, d, I)}


def _scale_buffer(rows, K):
    return torch.ones((_blocks(K), (rows + 3) // 4 * 4), dtype=torch.float32, device="cuda")


def _activations(g, rows, K, kind):
    """Rows of different sizes per channel, as activations have; of kind "blk" quantised, as a norm leaves them."""
    x = _normal(g, rows, K) * torch.exp(0.5 * _normal(g, K))
    if kind != "blk":
        return x.to(TYPES[kind])
    v, s = _block_quantise(x)
    scales = _scale_buffer(rows, K)
    scales[:, :rows] = s.t()
    return {"q": v.to(E4M3).view(torch.uint8), "s": scales}


def _routing(g, c):
    """Router logits N(0, 1) plus a fixed popularity of each expert; the top k's softmax weights, and the tables."""
    T, E, k, rows = c["T"], c["E"], c["k"], c["block_rows"]
    w, ids = (_normal(g, T, E) + 0.3 * _normal(g, E)).topk(k, dim=1)
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
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
    out = {"ids": ids, "counts": counts, "offsets": offsets, "perm": perm, "inv_perm": inv,
           "block_map": torch.where((b < tile_end[-1])[:, None], block_map, 0), "num_blocks": tile_end[-1:]}
    out = {n: v.to(torch.int32).contiguous() for n, v in out.items()}
    out["w"] = w.softmax(1)
    return out, int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    c, st = case, {"case": case}
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        st["x"] = _normal(g, T, d).to(TYPES[c["x"]])
        # a residual stream that several layers have added to, a few channels far larger than the others
        stream = 4 * _normal(g, T, d) * torch.exp(0.7 * _normal(g, d))
        st["residual"] = stream.to(TYPES[c["residual"]]) if c["residual"] != "none" else None
        st["gamma"] = (1 + 0.2 * _normal(g, d)).to(torch.bfloat16)
        st["eps"] = 1e-6
        st["stream"] = torch.empty_like(st["residual"]) if st["residual"] is not None else None
        st["y"] = torch.empty((T, d), dtype=TYPES[c["x"]], device="cuda") if c["y"] else None
        st["q"] = torch.empty((T, d), dtype=torch.uint8, device="cuda")
        st["s"] = _scale_buffer(T, d)
        st["values"] = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "quantize":
        E, N, K = c["E"], c["N"], c["K"]
        st["x"] = (_normal(g, E, N, K) * torch.exp(0.5 * _normal(g, K))).to(TYPES[c["x"]])
        if c["kind"] == "rows":
            st["x"] = st["x"].view(E * N, K)
            st["s"] = _scale_buffer(E * N, K)
        else:
            st["s"] = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float32, device="cuda")
        st["q"] = torch.empty(st["x"].shape, dtype=torch.uint8, device="cuda")
        st["values"] = torch.empty(st["x"].shape, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "linear":
        st["x"] = _activations(g, c["T"], c["K"], c["x"])
        st["weight"] = _matrix(g, 1, c["N"], c["K"])
        st["y"] = torch.empty((c["T"], c["N"]), dtype=TYPES[c["y"]], device="cuda")
    else:
        st["x"] = _activations(g, c["T"], c["d"], c["x"])
        st["routing"], st["capacity"] = _routing(g, c)  # capacity: the plain form's rows per expert
        st["routed"] = _experts(g, c["E"], c["d"], c["I"])
        st["shared"] = _experts(g, 1, c["d"], c["I_shared"]) if c["I_shared"] else None
        st["y"] = torch.empty((c["T"], c["d"]), dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ the plain form
def _power(a):
    """The least 2^e, e >= -126, with a <= 448 2^e = 1.75 2^(e + 8)."""
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1)
    return torch.ldexp(torch.ones_like(a), torch.where(a > 0, e - 9 + (m > 0.875).to(e.dtype), -126).clamp(min=-126))


def _block_quantise(x):
    """E4M3 values in units of the block's scale [..., K], and the scales [..., ceil(K/128)], 128 columns of a row."""
    b = _padded(x).view(*x.shape[:-1], -1, BLOCK)
    s = _power(b.abs().amax(-1))
    v = (b / s[..., None]).to(E4M3).float()
    return v.view(*x.shape[:-1], -1)[..., :x.shape[-1]], s


def _quantised(x):
    """x after a round trip through the 8-bit format."""
    v, s = _block_quantise(x)
    return v * s.repeat_interleave(BLOCK, -1)[..., :x.shape[-1]]


def _spread(s, N, K):
    return s.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def _weights(m):
    N, K = m["q"].shape[-2:]
    return m["q"].view(E4M3).float() * _spread(m["s"], N, K)


def _input(x):
    """The fp32 values of activations as the products take them."""
    if not isinstance(x, dict):
        return _quantised(x.float())
    rows, K = x["q"].shape
    return x["q"].view(E4M3).float() * x["s"][:, :rows].t().repeat_interleave(BLOCK, 1)[:, :K]


def _plain_norm(st):
    c = st["case"]
    r = st["x"].float()
    out = {}
    if st["residual"] is not None:
        out["residual"] = (r + st["residual"].float()).to(st["residual"].dtype)
        r = out["residual"].float()
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + st["eps"]) * st["gamma"].float()
    if c["y"]:
        out["y"] = y.to(st["x"].dtype)
    out["values"] = _quantised(y).to(torch.bfloat16)
    return out


def _plain_quantize(st):
    x = st["x"].float()
    if st["case"]["kind"] == "rows":
        return _quantised(x).to(torch.bfloat16)
    E, N, K = x.shape
    b = _padded(x, rows=True).view(E, _blocks(N), BLOCK, _blocks(K), BLOCK)
    s = _spread(_power(b.abs().amax((2, 4))), N, K)
    return ((x / s).to(E4M3).float() * s).to(torch.bfloat16)


def _ffn(x, ex):
    """x [E][C][d] fp32 through E experts."""
    gate = torch.matmul(x, _weights(ex["gate"]).transpose(1, 2))
    up = torch.matmul(x, _weights(ex["up"]).transpose(1, 2))
    h = _quantised(gate / (1 + torch.exp(-gate)) * up)
    return torch.matmul(h, _weights(ex["down"]).transpose(1, 2))


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
    c, r = st["case"], st["routing"]
    x = _input(st["x"])
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
    return y.to(torch.bfloat16)


def _plain(st):
    op = st["case"]["op"]
    if op == "norm":
        return _plain_norm(st)
    if op == "quantize":
        return _plain_quantize(st)
    if op == "linear":
        return torch.matmul(_input(st["x"]), _weights(st["weight"])[0].t()).to(TYPES[st["case"]["y"]])
    return _plain_layer(st)


# ------------------------------------------------------------------ the library's calls
def _handles(st):
    """The objects that a program keeps beside its tensors: they hold pointers to them and workspaces."""
    import bit_moe_expert_gb300 as bm
    c = st["case"]
    h = {"bm": bm}
    if c["op"] == "norm" or c["op"] == "quantize":
        h["out"] = (bm.BlkMat if c["op"] == "quantize" and c["kind"] == "weights" else bm.BlkAct)(st["q"], st["s"])
        return h
    h["x"] = bm.BlkAct(st["x"]["q"], st["x"]["s"]) if c["x"] == "blk" else st["x"]
    if c["op"] == "linear":
        h["w"] = bm.BlkMat(st["weight"]["q"], st["weight"]["s"])
        h["ws"] = bm.workspace(bm.moe_blk_linear_workspace_bytes(c["T"], c["N"], c["K"]))
    else:
        def experts(ex):
            return bm.BlkExperts(**{n: bm.BlkMat(m["q"], m["s"]) for n, m in ex.items()})

        h["routing"] = bm.Routing(**st["routing"], block_rows=c["block_rows"])
        h["routed"] = experts(st["routed"])
        h["shared"] = experts(st["shared"]) if st["shared"] is not None else None
        h["ws"] = bm.workspace(bm.moe_blk_forward_workspace_bytes(c["T"], c["d"], c["I"], c["E"], c["k"], c["I_shared"],
                                                                  c["block_rows"]))
    return h


def _kernels(st):
    c = st["case"]
    if "handles" not in st:
        st["handles"] = _handles(st)
    h = st["handles"]
    bm = h["bm"]
    if c["op"] == "norm":
        # the stream goes to memory of its own, so that every pass starts from the same
        bm.moe_rmsnorm(st["x"], st["gamma"], st["eps"], residual=st["residual"], stream_out=st["stream"], Y=st["y"],
                       out=h["out"])
        bm.moe_blk_dequant(h["out"], st["values"])
        out = {"values": st["values"]}
        if st["residual"] is not None:
            out["residual"] = st["stream"]
        if c["y"]:
            out["y"] = st["y"]
        return out
    if c["op"] == "quantize":
        (bm.moe_blk_quantize if c["kind"] == "rows" else bm.moe_blk_quantize_weights)(st["x"], h["out"])
        bm.moe_blk_dequant(h["out"], st["values"])
        return st["values"]
    if c["op"] == "linear":
        if c["x"] == "blk":
            bm.moe_blk_matmul(h["x"], h["w"], st["y"], h["ws"])
        else:
            bm.moe_blk_linear(h["x"], h["w"], st["y"], h["ws"])
        return st["y"]
    bm.moe_blk_forward(h["x"], h["routed"], h["shared"], h["routing"], st["y"], h["ws"])
    return st["y"]


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _matrix_bytes(N, K):
    return N * K + 4 * _blocks(N) * _blocks(K)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        stream = 0 if c["residual"] == "none" else 2 * BYTES[c["residual"]]
        return {"bytes": n * (BYTES[c["x"]] * (1 + c["y"]) + stream + 2) + 2 * c["d"], "flops": 8 * n}
    if c["op"] == "quantize":
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": n * (BYTES[c["x"]] + 2), "flops": 3 * n}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": T * K * BYTES[c["x"]] + _matrix_bytes(N, K) + T * N * BYTES[c["y"]], "flops": 2 * T * N * K}
    T, E, k, d = c["T"], c["E"], c["k"], c["d"]
    active = E * (1 - (1 - k / E) ** T)  # experts that some token takes, at about even popularity
    weights = active * (2 * _matrix_bytes(c["I"], d) + _matrix_bytes(d, c["I"]))
    if c["I_shared"]:
        weights += 2 * _matrix_bytes(c["I_shared"], d) + _matrix_bytes(d, c["I_shared"])
    return {"bytes": weights + T * d * (BYTES[c["x"]] + 2) + 16 * T * k,
            "flops": 6 * T * d * (k * c["I"] + c["I_shared"])}


# ------------------------------------------------------------------ in 64 bits
def _exact_scale(a):
    """fp64 magnitudes: the powers of two, from the definition's inequality itself."""
    e = torch.where(a > 0, torch.floor(torch.log2(a.clamp(min=1e-300))) - 9, torch.full_like(a, -126)).clamp(min=-126)
    for _ in range(3):
        e = e + (a > 448 * torch.exp2(e)).double()
    return torch.exp2(e)


def _exact_round(v):
    """fp64 -> the nearest E4M3 value: three mantissa bits, steps of 2^-9 below 2^-6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_rows(x):
    """fp64 [..., K] in blocks of 128 columns, block by block."""
    out = torch.empty_like(x)
    for k in range(0, x.shape[-1], BLOCK):
        b = x[..., k:k + BLOCK]
        s = _exact_scale(b.abs().amax(-1, keepdim=True))
        out[..., k:k + BLOCK] = _exact_round(b / s) * s
    return out


def _e4m3_values():
    """The 256 codes' values, from the format's fields."""
    v = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        a = math.nan if code & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-a if code >> 7 else a)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_weight(m):
    w = _e4m3_values()[m["q"].int()]
    n, k = (torch.arange(x, device="cuda") // BLOCK for x in w.shape[-2:])
    w *= m["s"].double()[:, n][:, :, k]
    return w


def _exact_input(x):
    if not isinstance(x, dict):
        return _exact_rows(x.double())
    rows, K = x["q"].shape
    return _e4m3_values()[x["q"].int()] * x["s"].double()[torch.arange(K, device="cuda") // BLOCK][:, :rows].t()


def _exact_ffn(x, ex):
    h = torch.bmm(x, _exact_weight(ex["gate"]).transpose(1, 2))
    h = h * torch.sigmoid(h) * torch.bmm(x, _exact_weight(ex["up"]).transpose(1, 2))
    return torch.bmm(_exact_rows(h), _exact_weight(ex["down"]).transpose(1, 2))


def _exact_norm(st):
    out = {}
    r = st["x"].double()
    if st["residual"] is not None:
        r = (r + st["residual"].double()).to(st["residual"].dtype).double()  # the stream holds what its type can hold
        out["residual"] = r
    y = r * (r.square().sum(1, keepdim=True) / r.shape[1] + st["eps"]).rsqrt() * st["gamma"].double()
    if st["case"]["y"]:
        out["y"] = y
    out["values"] = _exact_rows(y)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        return _exact_norm(st)
    if c["op"] == "quantize":
        x = st["x"].double()
        if c["kind"] == "rows":
            return _exact_rows(x)
        for n in range(0, c["N"], BLOCK):
            for k in range(0, c["K"], BLOCK):
                b = x[:, n:n + BLOCK, k:k + BLOCK]
                s = _exact_scale(b.abs().amax((1, 2), keepdim=True))
                x[:, n:n + BLOCK, k:k + BLOCK] = _exact_round(b / s) * s
        return x
    if c["op"] == "linear":
        return _exact_input(st["x"]) @ _exact_weight(st["weight"])[0].t()
    r = st["routing"]
    token, row = _rows_of(r, c, st["capacity"])
    x = _exact_input(st["x"])
    y = torch.zeros((c["T"], c["k"], c["d"]), dtype=torch.float64, device="cuda").view(-1, c["d"])
    for e0 in range(0, c["E"], 32):  # 32 experts at a time
        some = {n: {"q": m["q"][e0:e0 + 32], "s": m["s"][e0:e0 + 32]} for n, m in st["routed"].items()}
        part = _exact_ffn(x[token[e0:e0 + 32]], some).view(-1, c["d"])
        at = row - e0 * st["capacity"]
        mine = (at >= 0) & (at < part.shape[0])
        y[mine] = part[at[mine]]
    y = (y.view(c["T"], c["k"], c["d"]) * r["w"].double()[:, :, None]).sum(1)
    if st["shared"] is not None:
        y = y + _exact_ffn(x[None], st["shared"])[0]
    return y
