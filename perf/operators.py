"""The serving operators around the hybrid block, as a user calls them, with their plain forms.

Three operators and the calls between them:

  norm     h = x + residual; y = h rsqrt(mean(h^2) + eps) w; y as e4m3 codes with one scale for
           each 128 columns of a row (the operand of the product below), or as bf16 / float32;
  product  out = A W^T with A and W held as e4m3 codes, a scale for each 1 x 128 block of A and
           each 128 x 128 block of W; with "quantise" A arrives as bf16 and is quantised first;
  prefix   the full-attention layer for a batch whose sequences share one long prefix: every
           query attends to the shared rows and, causally, to its own sequence's rows.

`run` computes them in torch in 32 bits, or, with `own`, through the framework.
"""
import torch

own = False

DIM = 128                   # head size, and the length of a scale block
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 8 sequences in front of the block's projections: latency
        dict(name="norm decode 8x4096 e4m3", op="norm", rows=8, d=4096, res="bf16", out="e4m3"),
        # the residual stream of a 32k-token prompt: bandwidth
        dict(name="norm prefill 32768x4096 e4m3", op="norm", rows=32768, d=4096, res="bf16", out="e4m3"),
        # a float32 residual stream, a width that ends inside a scale block, both kinds of output
        dict(name="norm ragged 1023x4880 f32 residual", op="norm", rows=1023, d=4880, res="f32", out="both"),
        # the shared K/V head of one new token: the smallest product
        dict(name="product kv 1x256x4096", op="product", m=1, n=256, k=4096, out="bf16", quantise=False),
        # queries of a full layer and three sparse layers (32 heads each) for 8 decoding sequences
        dict(name="product queries 8x16384x4096", op="product", m=8, n=16384, k=4096, out="bf16", quantise=False),
        # attention outputs of two 512-token chunks, quantised and projected back
        dict(name="product output 1024x4096x4096", op="product", m=1024, n=4096, k=4096, out="bf16", quantise=True),
        # the full layer's queries of a 32k-token prompt: the largest product
        dict(name="product prefill 32768x4096x4096", op="product", m=32768, n=4096, k=4096, out="bf16", quantise=False),
        # no size a multiple of a tile, float32 result
        dict(name="product ragged 777x1000x2064 f32", op="product", m=777, n=1000, k=2064, out="f32", quantise=False),
        # two short requests behind a short system prompt: latency
        dict(name="prefix 2x1 behind 1000", op="prefix", batch=2, n_q=1, heads=16, prefix=1000, own_max=200, cache="bf16"),
        # 32 agents decoding behind one 128k-token context
        dict(name="prefix 32x1 behind 131072", op="prefix", batch=32, n_q=1, heads=32, prefix=131072, own_max=2048, cache="bf16"),
        # 16 agents behind a 64k-token context in an e4m3 cache
        dict(name="prefix 16x1 behind 65536 e4m3", op="prefix", batch=16, n_q=1, heads=32, prefix=65536, own_max=1024, cache="e4m3"),
        # four prompts' first chunks behind a shared context of odd length
        dict(name="prefix 4x128 behind 30001", op="prefix", batch=4, n_q=128, heads=32, prefix=30001, own_max=300, cache="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "product", "product", "prefix", "prefix"])
    if op == "norm":
        d = 16 * _spread(rng, 4, 1024)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(32768, 2 ** 27 // d))), d=d,
                    res=rng.choice(["none", "bf16", "f32"]), out=rng.choice(["bf16", "f32", "e4m3", "both"]))
    if op == "product":
        n, k = _spread(rng, 16, 16384), 16 * _spread(rng, 4, 1024)
        return dict(op=op, m=_spread(rng, 1, max(1, min(32768, 2 ** 38 // (n * k)))), n=n, k=k,
                    out=rng.choice(["bf16", "bf16", "f32"]), quantise=rng.random() < 0.3)
    heads, n_q, batch = rng.choice([16, 32]), rng.choice([1, 1, 1, _spread(rng, 2, 256)]), _spread(rng, 1, 64)
    batch = max(1, min(batch, 512 // n_q))
    most = 32 * 32 * 131072 // (batch * n_q * heads)
    return dict(op=op, batch=batch, n_q=n_q, heads=heads, prefix=_spread(rng, 1, min(131072, most)),
                own_max=n_q + _spread(rng, 1, 2048), cache=rng.choice(["bf16", "e4m3"]))


# ---------------------------------------------------------------- inputs

def _blocks(x):
    """x [rows, cols] in blocks of 128 columns, [rows, blocks, 128], zeros behind the last column."""
    rows, cols = x.shape
    nb = -(-cols // DIM)
    return torch.nn.functional.pad(x, (0, nb * DIM - cols)).view(rows, nb, DIM)


def _scale_buffer(blocks, rows):
    """Scales [column blocks, rows or row blocks]; a column block's scales start 16 bytes apart."""
    return torch.empty((blocks, -(-rows // 4) * 4), device="cuda")[:, :rows]


def _scale(amax):
    """amax / 448 in float32, one division (a division by a plain number would multiply by its rounded reciprocal)."""
    return torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))


def _to_codes(y):
    """e4m3 codes of y [rows, cols] with a scale for each 128 columns: (codes, scales [blocks, rows])."""
    b = _blocks(y)
    scale = _scale(b.abs().amax(-1))
    codes = (b / scale[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).flatten(1)[:, :y.shape[1]].contiguous().view(torch.float8_e4m3fn), scale.t()


def _weight_codes(w):
    """As _to_codes, with one scale for each 128 x 128 block."""
    n, k = w.shape
    nb, kb = -(-n // DIM), -(-k // DIM)
    t = torch.nn.functional.pad(w, (0, kb * DIM - k, 0, nb * DIM - n)).view(nb, DIM, kb, DIM)
    scale = _scale(t.abs().amax((1, 3)))
    codes = (t / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(nb * DIM, kb * DIM)[:n, :k].contiguous().view(torch.float8_e4m3fn), scale.t()


def _held(scale):
    """The scales in a buffer of the layout that the framework reads."""
    return _scale_buffer(*scale.shape).copy_(scale)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        # a residual stream: some channels are many times the others, as in trained models
        channel = torch.exp(normal(d))
        s["x"] = (normal(rows, d) * channel).bfloat16()
        s["res"] = None
        if case["res"] != "none":
            s["res"] = (2 * normal(rows, d) * channel).to(torch.bfloat16 if case["res"] == "bf16" else torch.float32)
            s["res_out"] = torch.empty_like(s["res"])
        s["w"] = (1 + 0.2 * normal(d)).bfloat16()
        s["y"] = s["codes"] = s["scales"] = None
        if case["out"] in ("bf16", "f32", "both"):
            s["y"] = torch.empty((rows, d), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device="cuda")
        if case["out"] in ("e4m3", "both"):
            s["codes"] = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = _scale_buffer(-(-d // DIM), rows)
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = (normal(m, k) * torch.exp(0.5 * normal(k))).bfloat16()
        codes, scale = _weight_codes(normal(n, k) / k ** 0.5)
        s["w"], s["w_scale"] = codes, _held(scale)
        if case["quantise"]:
            s["x"] = a
            s["a"] = torch.empty((m, k), dtype=torch.float8_e4m3fn, device="cuda")
            s["a_scale"] = _scale_buffer(-(-k // DIM), m)
        else:
            codes, scale = _to_codes(a.float())
            s["a"], s["a_scale"] = codes, _held(scale)
        s["out_"] = torch.empty((m, n), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device="cuda")
        s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
    else:
        b, n_q, heads, p = case["batch"], case["n_q"], case["heads"], case["prefix"]
        lens = torch.randint(n_q, case["own_max"] + 1, (b,), generator=g, device="cuda").tolist()
        # the prefix stands behind 37 rows of something else; the sequences follow it, with room to grow
        s["start"], at = [], 37 + p
        for t in lens:
            s["start"].append(at)
            at += t + 5
        s["prefix_start"], s["lens"] = 37, lens
        k, v = normal(at, DIM).bfloat16(), normal(at, DIM).bfloat16()
        s["k_scale"] = s["v_scale"] = None
        if case["cache"] == "e4m3":
            (k, ks), (v, vs) = _to_codes(k.float()), _to_codes(v.float())
            s["k_scale"], s["v_scale"] = ks[0].contiguous(), vs[0].contiguous()
        s["k"], s["v"] = k, v
        s["q"] = (1.5 * normal(b, n_q, heads, DIM)).bfloat16()
        s["out_"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, n_q, heads), device="cuda")
        s["own_start"] = torch.tensor(s["start"], device="cuda")
        s["own_len"] = torch.tensor(lens, device="cuda")
        if own:  # the geometry and the workspace, which a serving loop keeps
            import token_level_sparse_hs2_b200 as hs2
            s["cache_"] = hs2.KvCache(k, v, s["start"], lens, n_q, heads, s["k_scale"], s["v_scale"])
            s["ws"] = torch.empty(hs2.prefix_attn_workspace_size(s["cache_"], p), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm, "product": _product, "prefix": _prefix}[s["op"]](s)


def _run_own(s):
    import token_level_sparse_hs2_b200 as hs2
    if s["op"] == "norm":
        hs2.rms_norm(s["x"], s["w"], EPS, residual=s["res"], residual_out=s.get("res_out"), out=s["y"],
                     codes=s["codes"], scales=s["scales"])
        return _some(residual=s.get("res_out"), y=s["y"], codes=s["codes"], scales=s["scales"])
    if s["op"] == "product":
        if s["quantise"]:
            hs2.fp8_quantize(s["x"], s["a"], s["a_scale"])
        hs2.gemm_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out_"], s["ws"])
        return s["out_"]
    hs2.prefix_attn(s["cache_"], s["prefix_start"], s["prefix"], s["q"], s["out_"], s["lse"], s["ws"])
    return {"out": s["out_"], "lse": s["lse"]}


def _some(**outputs):
    return {name: t for name, t in outputs.items() if t is not None}


def _norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    codes, scales = _to_codes(y) if s["codes"] is not None else (None, None)
    return _some(residual=None if s["res"] is None else h.to(s["res"].dtype), y=None if s["y"] is None else y.to(s["y"].dtype),
                 codes=codes, scales=scales)


def _product(s):
    k = s["w"].shape[1]
    a, a_scale = _to_codes(s["x"].float()) if s["quantise"] else (s["a"], s["a_scale"])
    a = (_blocks(a.float()) * a_scale.t()[..., None]).flatten(1)[:, :k]
    w_scale = s["w_scale"].t().repeat_interleave(DIM, 0)[:s["w"].shape[0]]
    w = (_blocks(s["w"].float()) * w_scale[..., None]).flatten(1)[:, :k]
    return (a @ w.t()).to(s["out_"].dtype)


def _prefix(s):
    b, n_q, heads, _ = s["q"].shape
    p, p0 = s["prefix"], s["prefix_start"]
    q = s["q"].float().view(b, n_q * heads, DIM) / DIM ** 0.5
    k, v = s["k"].float(), s["v"].float()
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    # each sequence's own rows; a query sees those up to its own position
    t = torch.arange(max(s["lens"]), device="cuda")
    rows = s["own_start"][:, None] + torch.minimum(t, s["own_len"][:, None] - 1)
    last = s["own_len"][:, None] - n_q + torch.arange(n_q, device="cuda")
    seen = (t <= last[..., None]).repeat_interleave(heads, 1)
    x_prefix = q.view(-1, DIM) @ k[p0:p0 + p].t()
    x_own = (q @ k[rows].transpose(1, 2)).masked_fill(~seen, -torch.inf).flatten(0, 1)
    top = torch.maximum(x_prefix.amax(-1), x_own.amax(-1))[:, None]
    e_prefix, e_own = torch.exp(x_prefix - top), torch.exp(x_own - top)
    total = e_prefix.sum(-1) + e_own.sum(-1)
    o = e_prefix @ v[p0:p0 + p] + (e_own.view(b, n_q * heads, -1) @ v[rows]).flatten(0, 1)
    return {"out": (o / total[:, None]).view(b, n_q, heads, DIM).to(s["out_"].dtype),
            "lse": (torch.log(total) + top[:, 0]).view(b, n_q, heads)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["d"]
        per = 2 + {"none": 0, "bf16": 4, "f32": 8}[case["res"]] + {"bf16": 2, "f32": 4, "e4m3": 1, "both": 3}[case["out"]]
        scales = 4 * case["rows"] * -(-case["d"] // DIM) if case["out"] in ("e4m3", "both") else 0
        return {"bytes": n * per + 2 * case["d"] + scales, "flops": 6 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // DIM), -(-n // DIM)
        a = 2 * m * k if case["quantise"] else m * k + 4 * m * kb
        return {"bytes": a + n * k + 4 * nb * kb + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    b, n_q, heads, p = case["batch"], case["n_q"], case["heads"], case["prefix"]
    own_mean = (n_q + case["own_max"]) / 2
    row = 2 * DIM * 2 if case["cache"] == "bf16" else 2 * (DIM + 4)
    keys = p + own_mean - (n_q - 1) / 2
    return {"bytes": (p + b * own_mean) * row + b * n_q * heads * (2 * DIM * 2 + 4), "flops": 4 * DIM * b * n_q * heads * keys}


# ---------------------------------------------------------------- the definitions in 64 bits

def _e4m3(x):
    """The e4m3 value nearest to each float64 (ties to even, at most 448 in magnitude)."""
    e = torch.floor(torch.log2(x.abs().clamp_min(1e-300))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h += s["res"].double()
        y = h / torch.sqrt(h.square().sum(1) / case["d"] + EPS)[:, None] * s["w"].double()
        codes = scales = None
        if s["codes"] is not None:  # the quotients before their rounding to codes
            codes, scales = torch.empty_like(y), torch.empty((-(-case["d"] // DIM), case["rows"]), dtype=torch.float64, device="cuda")
            for j in range(scales.shape[0]):
                part = y[:, j * DIM:(j + 1) * DIM]
                scales[j] = part.abs().max(1).values / E4M3_MAX
                codes[:, j * DIM:(j + 1) * DIM] = part / scales[j][:, None]
        return _some(residual=None if s["res"] is None else h, y=None if s["y"] is None else y, codes=codes, scales=scales)
    if case["op"] == "product":
        a, w = (s["x"] if case["quantise"] else s["a"]).double(), s["w"].double()
        total = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for j in range(s["w_scale"].shape[0]):
            part = a[:, j * DIM:(j + 1) * DIM]
            if case["quantise"]:
                scale = (part.abs().max(1).values / E4M3_MAX).float().double()
                part = _e4m3((part / scale[:, None]).float().double())  # the code of the float32 quotient
            else:
                scale = s["a_scale"][j].double()
            block = part @ w[:, j * DIM:(j + 1) * DIM].t()
            rows = s["w_scale"][j].double().repeat_interleave(DIM)[:case["n"]]
            total += block * scale[:, None] * rows
        return total
    b, n_q, heads, p, p0 = case["batch"], case["n_q"], case["heads"], case["prefix"], s["prefix_start"]
    k, v = s["k"].double(), s["v"].double()
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
    out = torch.empty((b, n_q, heads, DIM), dtype=torch.float64, device="cuda")
    lse = torch.empty((b, n_q, heads), dtype=torch.float64, device="cuda")
    for i in range(b):
        first, t = s["start"][i], s["lens"][i]
        keys, values = torch.cat([k[p0:p0 + p], k[first:first + t]]), torch.cat([v[p0:p0 + p], v[first:first + t]])
        for at in range(0, n_q, 16):
            q = s["q"][i, at:at + 16].double()
            x = torch.einsum("qhd,td->qht", q, keys) / DIM ** 0.5
            for j in range(q.shape[0]):
                x[j, :, p + t - n_q + at + j + 1:] = -torch.inf
            lse[i, at:at + 16] = torch.logsumexp(x, -1)
            out[i, at:at + 16] = torch.einsum("qht,td->qhd", torch.exp(x - lse[i, at:at + 16, :, None]), values)
    return {"out": out, "lse": lse}
