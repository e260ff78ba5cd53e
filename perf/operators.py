"""Cases for measuring the gradient-norm and clipping operators.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes a case's inputs on
the GPU, ``run()`` makes one pass: with ``own`` the framework's calls, without
it the operators' plain form in torch.  ``exact()`` is the definition in 64
bits.

The operators (x_k: the tensors of a set, s: a scale, e.g. 1 / loss scale):
    norm        N = |s| * sqrt(sum of all x^2), or |s| * max |x|; the same for
                each tensor; c = s * min(1, max_norm / (N + 1e-6))
    clip        y_k = c * x_k, rounded to y_k's type
    code_norm   norm of tensors that are kept compressed
    momentum    m' = mu * m + c * g, w' = w - eta * m', with w and m kept
                compressed and c read on the device
    sgd         w' = w - (eta * c) * m, likewise

Weights and momentum are kept compressed by a program that uses the
framework, so for the last three operators ``prepare`` encodes them where
``own`` is true; the plain form works on the same values uncompressed.  The
updates' results are codes; each pass decodes them too, since a result is
compared by the values that it stands for.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
CODE = 1 + 25 * 256 * 4 / 65536 + 2 * 256 / 65536   # bytes an element takes in a CLEAN block


# ------------------------------------------------------------------ sizes

def layer_sizes():
    """The tensors of one layer of the Qwen3-4B-shaped set that the benchmark
    trains: projections and gated MLP, then the four norm vectors."""
    hid, ffn, nq, nkv, hd = 2560, 9728, 32, 8, 128
    return [hid * nq * hd, hid * nkv * hd, hid * nkv * hd, nq * hd * hid, hid * ffn, hid * ffn, ffn * hid,
            hid, hid, hd, hd]


def sizes_of(case):
    kind = case["set"]
    if kind == "layers":
        out = [151936 * 2560] if case["embed"] else []
        out += layer_sizes() * case["layers"]
        return out + ([2560] if case["embed"] else [])
    if kind == "vectors":
        return layer_sizes()[-4:] * case["layers"]
    if kind == "one":
        return [case["elems"]]
    # ragged: `count` tensors of about elems / count elements each, spread
    # over a factor of a hundred, odd sizes among them
    r = random.Random(case["elems"] * 1000003 + case["count"])
    w = [math.exp(r.uniform(0.0, math.log(100.0))) for _ in range(case["count"])]
    t = sum(w)
    return [max(1, int(case["elems"] * v / t)) for v in w]


def places(case):
    """(start of each tensor in its buffer, buffer length).  Ragged sets lie
    back to back, as views of one flat gradient buffer do (any alignment);
    the others start at multiples of 256 elements, as separate allocations."""
    at, out = 0, []
    for n in sizes_of(case):
        out.append(at)
        at += n if case["set"] == "ragged" and case["op"] in ("norm", "clip") else -(-n // 256) * 256
    return out, at


def parts(flat, case):
    return [flat[a:a + n] for a, n in zip(places(case)[0], sizes_of(case))]


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four norm vectors of one layer: the smallest call, all latency
        {"name": "norm-vectors-bf16", "op": "norm", "set": "vectors", "layers": 1, "dtype": "bf16", "kind": "l2",
         "max_norm": 1.0, "scale": 1.0},
        # fp16 gradients under a loss scale, largest magnitude (overflow watch), flat buffer views
        {"name": "norm-ragged-fp16-max", "op": "norm", "set": "ragged", "count": 61, "elems": 9_437_311,
         "dtype": "fp16", "kind": "max", "max_norm": 0.5, "scale": 1.0 / 1024},
        # fp32 accumulated gradients of a mid-sized model, flat buffer views
        {"name": "norm-ragged-fp32", "op": "norm", "set": "ragged", "count": 148, "elems": 162_201_601,
         "dtype": "fp32", "kind": "l2", "max_norm": 1.0, "scale": 0.125},
        # the whole benchmark set's bf16 gradients, 398 tensors
        {"name": "norm-set-bf16", "op": "norm", "set": "layers", "layers": 36, "embed": True, "dtype": "bf16",
         "kind": "l2", "max_norm": 1.0, "scale": 1.0},
        # a small model's fp16 gradients
        {"name": "clip-ragged-fp16", "op": "clip", "set": "ragged", "count": 23, "elems": 1_048_583,
         "dtype": "fp16", "to": "fp16", "coef": 0.37},
        # fp32 accumulators clipped into the bf16 buffers that the momentum step reads
        {"name": "clip-layers-fp32-bf16", "op": "clip", "set": "layers", "layers": 12, "embed": True,
         "dtype": "fp32", "to": "bf16", "coef": 0.0421},
        # one compressed tensor with a partial last block
        {"name": "code-norm-one", "op": "code_norm", "set": "one", "elems": 1_310_977, "kind": "l2",
         "max_norm": 0.1, "scale": 1.0},
        # the benchmark set's momentum, kept compressed
        {"name": "code-norm-set", "op": "code_norm", "set": "layers", "layers": 36, "embed": True, "kind": "l2",
         "max_norm": 1.0, "scale": 1.0},
        # one projection matrix
        {"name": "momentum-one", "op": "momentum", "set": "one", "elems": 2560 * 1024, "coef": 0.81, "mu": 0.9,
         "eta": 0.1},
        # a pipeline stage of eight layers
        {"name": "momentum-stage", "op": "momentum", "set": "layers", "layers": 8, "embed": False, "coef": 0.0733,
         "mu": 0.95, "eta": 0.2},
        {"name": "sgd-ragged", "op": "sgd", "set": "ragged", "count": 17, "elems": 7_340_033, "coef": 0.5,
         "eta": 0.5},
        {"name": "sgd-stage", "op": "sgd", "set": "layers", "layers": 8, "embed": False, "coef": 0.31, "eta": 0.3},
    ]


def draw(rng):
    op = rng.choice(["norm", "norm", "clip", "clip", "code_norm", "momentum", "sgd"])
    case = {"op": op}
    # total elements over five decades, odd sizes among them
    elems = int(math.exp(rng.uniform(math.log(3e3), math.log(4e8)))) | rng.choice([0, 1])
    if rng.random() < 0.25:
        case |= {"set": "layers", "layers": rng.randint(1, 6),
                 "embed": op in ("norm", "clip", "code_norm") and rng.random() < 0.3}
    elif op not in ("norm", "clip") and rng.random() < 0.3:
        case |= {"set": "one", "elems": elems}
    else:
        case |= {"set": "ragged", "count": rng.randint(1, max(1, min(300, elems // 500))), "elems": elems}
    if op == "norm":
        case |= {"dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "clip":
        case |= {"dtype": rng.choice(["bf16", "fp16", "fp32"])}
        case |= {"to": rng.choice([case["dtype"], "bf16"])}
    if op in ("norm", "code_norm"):
        case |= {"kind": rng.choice(["l2", "l2", "max"]), "max_norm": round(math.exp(rng.uniform(-5, 3)), 4),
                 "scale": rng.choice([1.0, 0.5, 1.0 / 256])}
    else:
        case |= {"coef": round(rng.uniform(0.01, 1.0), 4)}
    if op == "momentum":
        case |= {"mu": rng.choice([0.8, 0.9, 0.95])}
    if op in ("momentum", "sgd"):
        case |= {"eta": rng.choice([0.5, 0.1, 0.02])}
    return case


# ------------------------------------------------------------------ inputs

def values(case, seed, salt, sigma, dtype):
    """A flat buffer of N(0, sigma^2) values, with a thousandth of them about
    thirty times larger, as gradients have."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 8 + salt)
    n = places(case)[1]
    out = torch.empty(n, dtype=dtype, device="cuda")
    step = 1 << 28   # in pieces: the draw is in 32 bits
    at = 0
    while at < n:
        v = torch.randn(min(step, n - at), generator=g, device="cuda").mul_(sigma)
        if salt != 1:
            hit = torch.randint(0, v.numel(), (max(1, v.numel() // 1000),), generator=g, device="cuda")
            v[hit] = v[hit] * 30.0
        out[at:at + v.numel()] = v.to(dtype)
        at += v.numel()
    starts, _ = places(case)   # what lies between tensors is zero
    for a, k, b in zip(starts, sizes_of(case), starts[1:] + [n]):
        out[a + k:b] = 0
    return out


def inputs(case, seed):
    """The dense values of a case: {name: flat buffer}."""
    op = case["op"]
    if op in ("norm", "clip"):
        sigma = 1e-3 if case["dtype"] != "fp16" else 0.5   # fp16 gradients are under a loss scale
        return {"x": values(case, seed, 0, sigma, TYPES[case["dtype"]])}
    if op == "code_norm":
        return {"x": values(case, seed, 0, 1e-3, torch.bfloat16)}
    out = {"w": values(case, seed, 1, 0.02, torch.bfloat16), "m": values(case, seed, 2, 1e-3, torch.bfloat16)}
    if op == "momentum":
        out["g"] = values(case, seed, 3, 1e-3, torch.bfloat16)
    return out


def prepare(case, seed):
    s = {"case": case, **inputs(case, seed)}
    op = case["op"]
    if "coef" in case:
        s["coef"] = torch.tensor(case["coef"], dtype=torch.float32, device="cuda")
    if op == "clip":
        s["y"] = torch.zeros(places(case)[1], dtype=TYPES[case["to"]], device="cuda")
    if op in ("momentum", "sgd"):
        s["yw"] = torch.zeros_like(s["w"])
    if op == "momentum":
        s["ym"] = torch.zeros_like(s["m"])
    if own:
        keep(s, case)
    return s


def keep(s, case):
    """What a program that uses the framework keeps from step to step: the
    lists, the result buffers, and its operands as codes."""
    import lossless_bf16_tensor_split_amd as L
    s["L"] = L
    op, ns = case["op"], sizes_of(case)
    if op in ("norm", "clip"):
        s["xs"] = L.LctList(parts(s["x"], case))
        if op == "norm":
            s["out"] = L.alloc_norm(len(ns), each=True)
        else:
            s["ys"] = L.LctList(parts(s["y"], case))
        return
    lay = L.lct_layout_init(L.CLEAN)

    def group(sigma, dense):
        cb = L.lct_codebook_build(L.Model(L.GAUSSIAN, sigma, 0.0), dense[0])
        return L.LctGroup(ns, lay, [cb] * len(ns), dense)

    def coded(g):
        st = g.alloc_storage(sum(ns) // 8 + 65536)
        L.lct_encode_group(g, st)
        return st

    if op == "code_norm":
        s["g"] = group(1e-3, parts(s["x"], case))
        s["all"] = coded(s["g"])
        s["out"] = L.alloc_norm(len(ns), each=True, nblk=s["all"].sizes.nblk)
        return
    gw, gm = group(0.02, parts(s["w"], case)), group(1e-3, parts(s["m"], case))
    s["wc"], s["mc"] = coded(gw), coded(gm)
    cap = sum(ns) // 8 + 65536
    s["wo"] = gw.alloc_storage(cap)
    # bound to the buffers that the results are decoded into
    s["gw"], s["gm"] = group_to(L, gw, parts(s["yw"], case)), gm
    if op == "momentum":
        s["mo"] = gm.alloc_storage(cap)
        s["gm"] = group_to(L, gm, parts(s["ym"], case))
        s["gg"] = group_to(L, gm, parts(s["g"], case))


def group_to(L, g, dense):
    return L.LctGroup([int(v) for v in g.ns], g.layout, list(g.codebooks), dense)


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        L = s["L"]
        if op == "norm":
            out = s["out"]
            L.lct_list_norm(s["xs"], out, max_norm=case["max_norm"], scale=case["scale"],
                            kind=L.NORM_L2 if case["kind"] == "l2" else L.NORM_MAX)
            return {"norm": out.norm, "coef": out.coef, "each": out.each}
        if op == "clip":
            L.lct_list_clip(s["xs"], s["coef"], s["ys"])
            return {"y": s["y"]}
        if op == "code_norm":
            out = s["out"]
            L.lct_group_norm(s["g"], s["all"], out, max_norm=case["max_norm"], scale=case["scale"],
                             kind=L.NORM_L2 if case["kind"] == "l2" else L.NORM_MAX)
            return {"norm": out.norm, "coef": out.coef, "each": out.each}
        if op == "momentum":
            L.lct_momentum_step_clip_group(s["gw"], s["wc"], s["gm"], s["mc"], s["gg"], s["coef"], case["mu"],
                                           case["eta"], s["wo"], s["mo"])
            L.lct_decode_group(s["gw"], s["wo"])
            L.lct_decode_group(s["gm"], s["mo"])
            return {"w": s["yw"], "m": s["ym"]}
        L.lct_sgd_step_clip_group(s["gw"], s["wc"], s["gm"], s["mc"], case["eta"], s["coef"], s["wo"])
        L.lct_decode_group(s["gw"], s["wo"])
        return {"w": s["yw"]}
    if op in ("norm", "code_norm"):
        xs = parts(s["x"], case)
        if case["kind"] == "l2":
            # sums of squares in 64 bits: long sums of values that span decades
            sq = torch.stack([x.float().square().sum(dtype=torch.float64) for x in xs])
            each, total = sq.sqrt(), sq.sum().sqrt()
        else:
            each = torch.stack([x.float().abs().amax() for x in xs]).double()
            total = each.amax()
        each, total = each * abs(case["scale"]), total * abs(case["scale"])
        c = (case["max_norm"] / (total + EPS)).clamp(max=1.0) * case["scale"]
        return {"norm": total.float(), "coef": c.float(), "each": each.float()}
    if op == "clip":
        # the set lies in one buffer: one product over all of it
        s["y"].copy_((s["x"].float() * s["coef"]).to(s["y"].dtype))
        return {"y": s["y"]}
    if op == "momentum":
        m = (case["mu"] * s["m"].float() + s["coef"] * s["g"].float()).to(torch.bfloat16)
        w = (s["w"].float() - case["eta"] * m.float()).to(torch.bfloat16)
        s["yw"].copy_(w)
        s["ym"].copy_(m)
        return {"w": s["yw"], "m": s["ym"]}
    w = s["w"].float() - (case["eta"] * s["coef"]) * s["m"].float()
    s["yw"].copy_(w.to(torch.bfloat16))
    return {"w": s["yw"]}


def work(case):
    ns = sizes_of(case)
    n, k, op = sum(ns), len(ns), case["op"]
    if op == "norm":
        return {"bytes": n * BYTES[case["dtype"]] + 4 * k + 8, "flops": 2 * n}
    if op == "clip":
        return {"bytes": n * (BYTES[case["dtype"]] + BYTES[case["to"]]) + 4, "flops": n}
    if op == "code_norm":
        return {"bytes": n * CODE + 4 * k + 8, "flops": 2 * n}
    if op == "momentum":   # codes of w, m and the gradient in; codes and values of w', m' out
        return {"bytes": n * (2 * CODE + 2 + 2 * CODE + 4), "flops": 5 * n}
    return {"bytes": n * (2 * CODE + CODE + 2), "flops": 2 * n}


# ------------------------------------------------------------------ definition

def exact(case, seed):
    """The definition in float64.  Where padding lies between tensors its
    values are left out of the norms by summing tensor by tensor; elementwise
    results are given for whole buffers with the padding as run() leaves it."""
    op = case["op"]
    d = inputs(case, seed)
    if op in ("norm", "code_norm"):
        each = []
        for x in parts(d["x"], case):
            big = x.double().abs().max()
            if case["kind"] == "max":
                each.append(big)
            else:   # relative to the largest value, in slices
                each.append(big * sum((v.double() / big).pow(2).sum() for v in x.split(1 << 26)).sqrt())
        each = torch.stack(each)
        total = each.max() if case["kind"] == "max" else each.pow(2).sum().sqrt()
        each, total = each * abs(case["scale"]), total * abs(case["scale"])
        c = case["scale"] * torch.minimum(torch.ones_like(total), case["max_norm"] / (total + EPS))
        return {"norm": total, "coef": c, "each": each}
    # the coefficient as the float32 number that it is held in
    c = torch.tensor(case["coef"], dtype=torch.float32).double().item() if "coef" in case else None
    if op == "clip":
        return {"y": d["x"].double() * c}
    if op == "momentum":
        m = d["m"].double() * case["mu"] + d["g"].double() * c
        held = m.to(torch.float32).to(torch.bfloat16).double()   # the stored momentum is what moves the weights
        return {"w": d["w"].double() - held * case["eta"], "m": m}
    return {"w": d["w"].double() - d["m"].double() * (case["eta"] * c)}
