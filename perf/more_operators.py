"""Cases for measuring orthogonalised updates and token tables that stay compressed.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes a case's inputs on
the GPU, ``run()`` makes one pass: with ``own`` the framework's calls, without
it the operators' plain form in torch.  ``exact()`` is the definition in 64
bits.

The operators:
    ortho   y_k = s_k * NS(x_k) for every matrix of a list: x / (|x| + 1e-7),
            then `steps` times x <- a x + b (x x') x + c (x x')^2 x, which
            drives the singular values towards one (a tall matrix is taken
            transposed)
    mix     y' = a * y + (b * c) * x, y kept compressed, x dense, c read on the
            device; with `dense` a dense result too: y' itself, or looked ahead
            (Nesterov), a * y' + (b * c) * x
    rows    y_t = s * W[i_t], W kept compressed; an index outside the table
            (a padding token's) gives zeros
    grad    G[v] = s * sum of dy_t over the t with i_t = v, dense; added to
            what G holds with `add`

A program keeps weights, momentum and token table compressed, so for mix and
rows ``prepare`` encodes them where ``own`` is true; the plain form works on
the same values uncompressed.  The mix's results are codes; each pass decodes
them too, since a result is compared by the values that it stands for.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
CODE = 1 + 25 * 256 * 4 / 65536 + 2 * 256 / 65536   # bytes an element takes in a CLEAN block
COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ------------------------------------------------------------------ sizes

# (rows, columns) of the matrices of one layer of the Qwen3-4B-shaped set that
# the benchmark trains: query, key, value, output, gate, up, down
LAYER = [(2560, 4096), (2560, 1024), (2560, 1024), (4096, 2560), (2560, 9728), (2560, 9728), (9728, 2560)]
# and of the attention of one layer of the 162M-parameter set: qkv, output
SMALL = [(768, 2304), (768, 768)]


def shapes_of(case):
    """The matrices of an ortho case."""
    kind = case["set"]
    if kind == "layer":
        return LAYER * case["layers"]
    if kind == "attention":
        return SMALL * case["layers"]
    if kind == "one":
        return [(case["m"], case["n"])]
    # ragged: sides over a factor of sixteen up to `side`, odd ones among them
    r = random.Random(case["side"] * 1000003 + case["count"])
    side = lambda: max(1, int(case["side"] / math.exp(r.uniform(0.0, math.log(16.0)))))  # noqa: E731
    return [(side(), side()) for _ in range(case["count"])]


def sizes_of(case):
    """The tensors of a mix case."""
    kind = case["set"]
    if kind == "layers":
        return [m * n for m, n in LAYER] * case["layers"]
    if kind == "one":
        return [case["elems"]]
    r = random.Random(case["elems"] * 1000003 + case["count"])
    w = [math.exp(r.uniform(0.0, math.log(100.0))) for _ in range(case["count"])]
    t = sum(w)
    return [max(1, int(case["elems"] * v / t)) for v in w]


def places(ns):
    """(start of each tensor in one buffer, its length): starts at multiples of 256."""
    at, out = 0, []
    for n in ns:
        out.append(at)
        at += -(-n // 256) * 256
    return out, at


def parts(flat, ns):
    return [flat[a:a + n] for a, n in zip(places(ns)[0], ns)]


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the matrices of a toy model: launches and short products
        {"name": "ortho-ragged-small", "op": "ortho", "set": "ragged", "count": 9, "side": 259, "dtype": "bf16",
         "steps": 5, "scale": "one"},
        # one odd fp32 matrix (an accumulated gradient), taller than wide
        {"name": "ortho-odd-fp32", "op": "ortho", "set": "one", "m": 2049, "n": 777, "dtype": "fp32", "steps": 5,
         "scale": "rms"},
        # the attention matrices of the 162M-parameter set: many alike
        {"name": "ortho-attention-bf16", "op": "ortho", "set": "attention", "layers": 12, "dtype": "bf16", "steps": 5,
         "scale": "rms"},
        # one layer of the benchmark's set
        {"name": "ortho-layer-bf16", "op": "ortho", "set": "layer", "layers": 1, "dtype": "bf16", "steps": 5,
         "scale": "rms"},
        # one projection's weights: decay and an orthogonal update
        {"name": "mix-one", "op": "mix", "set": "one", "elems": 2560 * 1024, "a": 0.999, "b": -0.02, "coef": 1.0,
         "dense": "none"},
        # momentum of ragged tensors, its value wanted dense
        {"name": "mix-ragged-value", "op": "mix", "set": "ragged", "count": 17, "elems": 7_340_033, "a": 0.9, "b": 1.0,
         "coef": 0.43, "dense": "value"},
        # momentum of a pipeline stage of eight layers, looked ahead for the orthogonalisation
        {"name": "mix-stage-ahead", "op": "mix", "set": "layers", "layers": 8, "a": 0.95, "b": 1.0, "coef": 0.81,
         "dense": "ahead"},
        # one token of a decoding step
        {"name": "rows-token", "op": "rows", "rows": 151936, "cols": 2560, "tokens": 1, "draw": "flat", "dtype": "bf16",
         "scale": 1.0},
        # a training batch's tokens, frequent ones often
        {"name": "rows-batch", "op": "rows", "rows": 151936, "cols": 2560, "tokens": 8192, "draw": "zipf",
         "dtype": "bf16", "scale": 50.5964},
        # a smaller table, long batch, fp32 result
        {"name": "rows-small-fp32", "op": "rows", "rows": 50304, "cols": 768, "tokens": 16385, "draw": "zipf",
         "dtype": "fp32", "scale": 1.0},
        # a few tokens' fp32 gradient added to an fp32 table gradient (the head's, with tied weights)
        {"name": "grad-add-fp32", "op": "grad", "rows": 4001, "cols": 331, "tokens": 777, "draw": "zipf",
         "dtype": "fp32", "to": "fp32", "scale": 1.0, "add": True},
        # a training batch's gradient of the whole table, as the momentum step reads it
        {"name": "grad-batch", "op": "grad", "rows": 151936, "cols": 2560, "tokens": 16384, "draw": "zipf",
         "dtype": "bf16", "to": "bf16", "scale": 50.5964, "add": False},
    ]


def spread(rng, lo, hi):
    """A whole number over the logarithm of a range, odd or even."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) | rng.choice([0, 1])))


def draw(rng):
    op = rng.choice(["ortho", "ortho", "mix", "mix", "rows", "rows", "grad", "grad"])
    case = {"op": op}
    if op == "ortho":
        if rng.random() < 0.5:
            case |= {"set": "one", "m": spread(rng, 16, 6000), "n": spread(rng, 16, 6000)}
        else:
            case |= {"set": "ragged", "count": rng.randint(2, 24), "side": spread(rng, 64, 2600)}
        return case | {"dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "steps": rng.choice([5, 5, 4, 6]),
                       "scale": rng.choice(["one", "rms"])}
    if op == "mix":
        elems = spread(rng, 3000, 400_000_000)
        if rng.random() < 0.3:
            case |= {"set": "one", "elems": elems}
        else:
            case |= {"set": "ragged", "count": rng.randint(1, max(1, min(200, elems // 500))), "elems": elems}
        if rng.random() < 0.5:
            case |= {"a": rng.choice([0.9, 0.95]), "b": 1.0, "dense": rng.choice(["value", "ahead"])}
        else:
            case |= {"a": rng.choice([1.0, 0.999, 0.99]), "b": -rng.choice([0.02, 0.1]), "dense": "none"}
        return case | {"coef": round(rng.uniform(0.05, 1.0), 4)}
    cols = spread(rng, 33, 2560)
    rows = spread(rng, 300, min(151936, 160_000_000 // cols))
    case |= {"rows": rows, "cols": cols, "tokens": spread(rng, 1, 16384), "draw": rng.choice(["zipf", "zipf", "flat"]),
             "dtype": rng.choice(["bf16", "bf16", "fp32"]), "scale": rng.choice([1.0, 8.5])}
    if op == "grad":
        case |= {"to": rng.choice(["bf16", "fp32"]), "add": rng.random() < 0.4}
    return case


# ------------------------------------------------------------------ inputs

def source(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 8 + salt)
    return g


def normal(g, n, sigma, dtype):
    """N(0, sigma^2) values, drawn in pieces in 32 bits."""
    out = torch.empty(n, dtype=dtype, device="cuda")
    for at in range(0, n, 1 << 28):
        m = min(1 << 28, n - at)
        out[at:at + m] = torch.randn(m, generator=g, device="cuda").mul_(sigma).to(dtype)
    return out


def matrix(g, m, n, dtype):
    """A gradient's momentum: a few strong directions over noise."""
    r = min(8, m, n)
    x = torch.randn(m, r, generator=g, device="cuda") @ torch.randn(r, n, generator=g, device="cuda")
    x = x.mul_(0.5).add_(torch.randn(m, n, generator=g, device="cuda"))
    return x.mul_(1e-3 if dtype != torch.float16 else 0.5).to(dtype)


def indices(g, case):
    """Token numbers: all alike likely, or the k-th about 1 / k as likely as the
    first; a fiftieth of a longer batch is padding."""
    t, rows = case["tokens"], case["rows"]
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
    k = u * rows if case["draw"] == "flat" else torch.exp(u * math.log(rows + 1.0)) - 1.0
    k = k.to(torch.int64).clamp_(0, rows - 1)
    if t >= 64:
        k = torch.where(torch.rand(t, generator=g, device="cuda") < 0.02, torch.full_like(k, -1), k)
    return k


def inputs(case, seed):
    op = case["op"]
    if op == "ortho":
        g = source(seed, 0)
        return {"xs": [matrix(g, m, n, TYPES[case["dtype"]]) for m, n in shapes_of(case)]}
    if op == "mix":
        n = places(sizes_of(case))[1]
        big = case["dense"] == "none"   # weights and an update, or momentum and a gradient
        return {"y": normal(source(seed, 1), n, 0.02 if big else 1e-3, torch.bfloat16),
                "x": normal(source(seed, 2), n, 0.02 if big else 1e-3, torch.bfloat16)}
    out = {"index": indices(source(seed, 3), case)}
    if op == "rows":
        out["w"] = normal(source(seed, 4), case["rows"] * case["cols"], 0.02, torch.bfloat16)
    else:
        out["dy"] = normal(source(seed, 5), case["tokens"] * case["cols"], 1e-3, TYPES[case["dtype"]])
        out["dy"] = out["dy"].view(case["tokens"], case["cols"])
        if case["add"]:
            out["g"] = normal(source(seed, 6), case["rows"] * case["cols"], 1e-3, TYPES[case["to"]])
            out["g"] = out["g"].view(case["rows"], case["cols"])
    return out


def scales(case):
    """s_k: one, or the factor that gives an orthogonal update a usual root mean square."""
    return [1.0 if case["scale"] == "one" else 0.2 * math.sqrt(max(m, n)) for m, n in shapes_of(case)]


def prepare(case, seed):
    s = {"case": case, **inputs(case, seed)}
    op = case["op"]
    if op == "ortho":
        s["ys"] = [torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for m, n in shapes_of(case)]
        s["scales"] = scales(case)
    elif op == "mix":
        s["coef"] = torch.tensor(case["coef"], dtype=torch.float32, device="cuda")
        s["v"] = torch.zeros_like(s["y"])
        s["u"] = torch.zeros_like(s["x"])
    elif op == "rows":
        s["out"] = torch.empty(case["tokens"], case["cols"], dtype=TYPES[case["dtype"]], device="cuda")
    else:
        s["out"] = torch.empty(case["rows"], case["cols"], dtype=TYPES[case["to"]], device="cuda")
    if own:
        keep(s, case)
    return s


def keep(s, case):
    """What a program that uses the framework keeps from step to step: lists,
    working memory, and its operands as codes."""
    import lossless_bf16_tensor_split_amd as L
    s["L"] = L
    op = case["op"]
    if op == "ortho":
        s["xl"], s["yl"] = L.LctMatrices(s["xs"]), L.LctMatrices(s["ys"])
        s["work"] = L.alloc_orthogonal(s["xl"])
    elif op == "mix":
        # each member with the padding behind it, over which the plain form goes too
        lay, ns = L.lct_layout_init(L.CLEAN), [-(-n // 256) * 256 for n in sizes_of(case)]
        sigma = 0.02 if case["dense"] == "none" else 1e-3
        cb = L.lct_codebook_build(L.Model(L.GAUSSIAN, sigma, 0.0), s["y"])
        bind = lambda t: L.LctGroup(ns, lay, [cb] * len(ns), parts(t, ns))  # noqa: E731
        g, cap = bind(s["y"]), sum(ns) // 8 + 65536
        s["yc"], s["oc"] = g.alloc_storage(cap), g.alloc_storage(cap)
        L.lct_encode_group(g, s["yc"])
        # bound to the buffer that the result is decoded into
        s["gv"], s["gx"], s["gu"] = bind(s["v"]), bind(s["x"]), bind(s["u"])
    elif op == "rows":
        lay = L.lct_layout_init(L.CLEAN)
        s["cb"] = L.lct_codebook_build(L.Model(L.GAUSSIAN, 0.02, 0.0), s["w"])
        s["t"] = L.encode(s["cb"], s["w"], lay, s["w"].numel() // 8 + 65536)
        s["work"] = L.alloc_rows(case["tokens"])
    else:
        s["work"] = L.alloc_rows(case["tokens"], cols=case["cols"])


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        L = s["L"]
        if op == "ortho":
            L.lct_list_orthogonalize(s["xl"], s["yl"], s["work"], steps=case["steps"], coef=COEF, scale=s["scales"])
            return {"y": s["ys"]}
        if op == "mix":
            dense = s["gu"] if case["dense"] != "none" else None
            L.lct_mix_step_group(s["gv"], s["yc"], case["a"], s["gx"], case["b"], s["oc"], coef=s["coef"], dense=dense,
                                 ahead=case["dense"] == "ahead")
            L.lct_decode_group(s["gv"], s["oc"])
            return {"y": s["v"], "u": s["u"]} if dense is not None else {"y": s["v"]}
        if op == "rows":
            L.lct_tensor_rows(s["cb"], s["t"], s["index"], s["out"], s["work"], scale=case["scale"])
            return {"y": s["out"]}
        if case["add"]:
            # a program adds to the gradient that it has; a fresh copy here, so that passes are alike
            s["out"].copy_(s["g"])
        L.lct_rows_grad(s["index"], s["dy"], s["out"], s["work"], scale=case["scale"], add=case["add"])
        return {"g": s["out"]}
    if op == "ortho":
        return {"y": [plain_ortho(x, case["steps"], k) for x, k in zip(s["xs"], s["scales"])]}
    if op == "mix":
        bx = (case["b"] * s["coef"]) * s["x"].float()
        v = (case["a"] * s["y"].float() + bx).to(torch.bfloat16)
        if case["dense"] == "none":
            return {"y": v}
        return {"y": v, "u": (case["a"] * v.float() + bx).to(torch.bfloat16) if case["dense"] == "ahead" else v}
    inside = (s["index"] >= 0) & (s["index"] < case["rows"])
    at = torch.where(inside, s["index"], torch.zeros_like(s["index"]))
    if op == "rows":
        y = s["w"].view(case["rows"], case["cols"])[at].float() * case["scale"]
        return {"y": torch.where(inside[:, None], y, torch.zeros_like(y)).to(s["out"].dtype)}
    d = s["dy"].float() * case["scale"]
    d = torch.where(inside[:, None], d, torch.zeros_like(d))
    g = s["g"].float() if case["add"] else torch.zeros(case["rows"], case["cols"], device="cuda")
    return {"g": g.index_add(0, at, d).to(s["out"].dtype)}


def plain_ortho(x, steps, scale):
    a, b, c = COEF
    tall = x.shape[0] > x.shape[1]
    v = x.float().T if tall else x.float()
    v = v / (torch.sqrt((v * v).sum()) + EPS)
    for _ in range(steps):
        p = v @ v.T
        v = a * v + (b * p + c * (p @ p)) @ v
    return (scale * (v.T if tall else v)).to(torch.bfloat16).contiguous()


def work(case):
    op = case["op"]
    if op == "ortho":
        n = sum(m * k for m, k in shapes_of(case))
        flops = 0
        for m, k in shapes_of(case):   # x x' and its square are symmetric: half of each
            m, k = min(m, k), max(m, k)
            flops += case["steps"] * (m * m * k + m ** 3 + 2 * m * m * k)
        return {"bytes": n * (BYTES[case["dtype"]] + 2), "flops": flops}
    if op == "mix":   # codes and x in; codes, their values and a dense result out
        n = sum(sizes_of(case))
        return {"bytes": n * (2 * CODE + 4 + (0 if case["dense"] == "none" else 2)), "flops": 3 * n}
    t, rows, cols = case["tokens"], case["rows"], case["cols"]
    if op == "rows":   # the rows' own codes, once each at most
        return {"bytes": 8 * t + cols * (min(t, rows) * CODE + t * BYTES[case["dtype"]]), "flops": t * cols}
    touched = min(t, rows) if case["add"] else 0
    return {"bytes": 8 * t + cols * (t * BYTES[case["dtype"]] + (rows + touched) * BYTES[case["to"]]),
            "flops": t * cols}


# ------------------------------------------------------------------ definition

def exact(case, seed):
    op = case["op"]
    d = inputs(case, seed)
    if op == "ortho":
        a, b, c = COEF
        out = []
        for x, k in zip(d["xs"], scales(case)):
            # by columns where it is tall: (x' x) on the right instead of a transposed copy
            v = x.double()
            v = v / (v.norm() + EPS)
            for _ in range(case["steps"]):
                if v.shape[0] > v.shape[1]:
                    q = torch.mm(v.T, v)
                    v = a * v + b * torch.mm(v, q) + c * torch.mm(torch.mm(v, q), q)
                else:
                    q = torch.mm(v, v.T)
                    v = a * v + b * torch.mm(q, v) + c * torch.mm(q, torch.mm(q, v))
            out.append(k * v)
        return {"y": out}
    # device numbers as the float32 that they are held in
    held = lambda v: torch.tensor(v, dtype=torch.float32).double().item()  # noqa: E731
    if op == "mix":
        bx = d["x"].double() * (case["b"] * held(case["coef"]))
        v = d["y"].double() * case["a"] + bx
        if case["dense"] == "none":
            return {"y": v}
        kept = v.to(torch.float32).to(torch.bfloat16).double()   # the stored value is what is looked ahead from
        return {"y": v, "u": kept * case["a"] + bx if case["dense"] == "ahead" else v}
    rows, cols = case["rows"], case["cols"]
    inside = (d["index"] >= 0) & (d["index"] < rows)
    at = d["index"].clamp(0, rows - 1)
    if op == "rows":
        y = d["w"].view(rows, cols).index_select(0, at).double() * case["scale"]
        y[~inside] = 0
        return {"y": y}
    g = d["g"].double() if case["add"] else torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    dy = d["dy"].double()[inside] * case["scale"]
    # by sorted tokens: differences of the running sum at the ends of each token's run
    key, order = torch.sort(at[inside], stable=True)
    if key.numel():
        which, count = torch.unique_consecutive(key, return_counts=True)
        total = torch.zeros(which.numel(), cols, dtype=torch.float64, device="cuda")
        run_of = torch.repeat_interleave(torch.arange(which.numel(), device="cuda"), count)
        total.index_add_(0, run_of, dy[order])
        g[which] += total
    return {"g": g}
