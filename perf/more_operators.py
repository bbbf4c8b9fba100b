"""Cases of the routed layer's training operators, measured against their plain forms.

The operators between a router and a caller's own step through the experts,
and their gradients:

``dispatch``      tokens sorted by expert: offsets, the order and its inverse, and
                  the tokens' rows in that order
``combine``       back again with the routing weights applied
``combine_grad``  its gradient: the rows', and the weights'
``matmul``        the grouped product of bf16 rows and weights (``y``), the
                  gradient of its rows (``dx``) and of its weights (``dw``)
``swiglu``        silu(gate) * up, with gate and up kept in 8 bits
``swiglu_grad``   its gradient from the 8-bit checkpoint, with h again
``select_grad``   the gradient of the experts' selection to the router's logits

``own`` false: plain torch operations; ``own`` true: the library's kernels.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100  # smallest block maximum that a scale is made from
F8 = torch.float8_e4m3fn
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2, "fp8": 1}


def listed():
    return [
        # one decoded token sent to its experts
        dict(name="dispatch-decode", op="dispatch", T=1, H=2048, E=256, k=8, x="bf16", empty=0.0),
        # a long pass of the wide layer, some slots dropped
        dict(name="dispatch-long", op="dispatch", T=8192, H=4096, E=384, k=6, x="bf16", empty=0.02),
        # the experts' outputs of a prefill chunk, summed with their weights
        dict(name="combine-chunk", op="combine", T=2048, H=2048, k=8, dtype="bf16", weights=True, empty=0.0),
        # backward through the same step of a long pass of the wide layer
        dict(name="combine-grad-long", op="combine_grad", T=8192, H=4096, k=6, dtype="bf16", weights=True,
             empty=0.02),
        # a verify block of six tokens: 48 rows, most of them alone with their expert
        dict(name="matmul-verify", op="matmul", way="y", M=48, N=768, K=2048, G=256, skew=0.0, tail=0,
             out="bf16", add=False),
        # backward to the rows of a training chunk, Zipf-skewed, dropped rows behind the last group
        dict(name="matmul-dx-chunk-zipf", op="matmul", way="dx", M=16384, N=768, K=2048, G=256, skew=1.0,
             tail=37, out="bf16", add=False),
        # backward to the experts' weights, added to the fp32 gradients of the step's earlier chunks
        dict(name="matmul-dw-chunk", op="matmul", way="dw", M=16384, N=768, K=2048, G=256, skew=0.0, tail=0,
             out="f32", add=True),
        # a shared projection of a long pass: bound by the matrix cores
        dict(name="matmul-long", op="matmul", way="y", M=8192, N=4096, K=4096, G=1, skew=0.0, tail=0,
             out="bf16", add=False),
        # the activation of a training chunk with its 8-bit checkpoint
        dict(name="swiglu-chunk", op="swiglu", R=16384, I=768, dtype="bf16", keep=True, tail=0),
        # its gradient in a long pass of the wide layer, from the checkpoint
        dict(name="swiglu-grad-long", op="swiglu_grad", R=49152, I=2048, dtype="bf16", keep=True, tail=983),
        # a training chunk routed by softmax over bf16 logits
        dict(name="select-grad-chunk", op="select_grad", T=2048, E=256, k=8, score="softmax", renorm=True,
             scale=1.0, logits="bf16", balance=False),
        # a long pass routed by sigmoid scores, with a balance loss
        dict(name="select-grad-long", op="select_grad", T=8192, E=384, k=6, score="sigmoid", renorm=True,
             scale=2.5, logits="f32", balance=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "matmul", "matmul", "matmul", "swiglu", "swiglu_grad",
                     "select_grad"])
    if op in ("dispatch", "combine", "combine_grad"):
        H = _log(rng, 64, 4096)
        if rng.random() < 0.6:
            H = -(-H // 64) * 64
        E = rng.choice([4, 8, 16, 64, 128, 256, 384])
        k = rng.randint(1, min(10, E))
        T = _log(rng, 1, max(1, min(16384, 200_000_000 // (k * H * 2))))
        empty = rng.choice([0.0, 0.0, 0.1])
        if op == "dispatch":
            return dict(op=op, T=T, H=H, E=E, k=k, x=rng.choice(["bf16", "f32", "fp8"]), empty=empty)
        return dict(op=op, T=T, H=H, k=k, dtype=rng.choice(["bf16", "f32"]), weights=rng.random() < 0.7, empty=empty)
    if op == "matmul":
        N, K = _log(rng, 48, 4096), _log(rng, 48, 4096)
        if rng.random() < 0.7:
            N, K = -(-N // 8) * 8, -(-K // 8) * 8
        G = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(256, 300_000_000 // (N * K))))
        M = _log(rng, 1, 16384 if G > 1 else 8192)
        return dict(op=op, way=rng.choice(["y", "dx", "dw"]), M=M, N=N, K=K, G=G,
                    skew=rng.choice([0.0, 1.0]) if G > 1 else 0.0,
                    tail=rng.randint(0, M // 50) if G > 1 else 0, out=rng.choice(["bf16", "f32"]),
                    add=rng.random() < 0.4)
    if op in ("swiglu", "swiglu_grad"):
        I = _log(rng, 64, 4096)
        if rng.random() < 0.6:
            I = -(-I // 64) * 64
        R = _log(rng, 1, max(1, min(49152, 90_000_000 // I)))
        return dict(op=op, R=R, I=I, dtype=rng.choice(["bf16", "f32"]), keep=rng.random() < 0.7,
                    tail=rng.randint(0, R // 20))
    E = rng.randint(4, 512)
    return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(10, E)),
                score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                logits=rng.choice(["f32", "bf16"]), balance=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------

def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, shape, dtype, size=1.0):
    """Normal draws, made in parts so that no fp32 copy of a large bank is held."""
    out = torch.empty(shape, dtype=TORCH[dtype], device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, device="cuda", generator=g) * size
    return out


def _routing(g, T, E, k, empty):
    """Distinct experts per token, some slots empty."""
    idx = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    drop = torch.rand(T, k, device="cuda", generator=g) < empty
    return torch.where(drop, -1, idx).contiguous()


def _sizes(case):
    """Rows of each group, largest first: equal or Zipf shares of all rows but the tail."""
    M, G = case["M"] - case["tail"], case["G"]
    if case["skew"] == 0.0:
        return [M // G + (i < M % G) for i in range(G)]
    share = [(i + 1) ** -case["skew"] for i in range(G)]
    s = sum(share)
    n = [int(M * v / s) for v in share]
    n[0] += M - sum(n)
    return n


def _quant(x):
    """(codes, scales) of rows: one scale for each 1 x 128 block.  Products by 448 before the division: a
    quotient half way between two codes then stays half way."""
    R, K = x.shape
    p = torch.zeros(R, _padded(K), device=x.device)
    p[:, :K] = x
    p = p.view(R, -1, BLOCK)
    top = p.abs().amax(2).clamp(min=TINY)
    return (p * E4M3_MAX / top[:, :, None]).to(F8).view(R, -1), top / E4M3_MAX


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, op=op)
    if op == "dispatch":
        T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
        out = "bf16" if case["x"] == "fp8" else case["x"]
        s["x"], s["sx"] = _randn(g, (T, H), out), None
        if case["x"] == "fp8":
            s["x"], s["sx"] = _quant(s["x"].float())
        s["idx"] = _routing(g, T, E, k, case["empty"])
        s["rows"] = torch.zeros(T * k, H, dtype=TORCH[out], device="cuda")
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["row_src"] = torch.zeros(T * k, dtype=torch.int32, device="cuda")
        s["row_of"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    elif op in ("combine", "combine_grad"):
        T, H, k, dtype = (case[n] for n in ("T", "H", "k", "dtype"))
        s["rows"] = _randn(g, (T * k, H), dtype)
        order = torch.randperm(T * k, device="cuda", generator=g).to(torch.int32).view(T, k)
        drop = torch.rand(T, k, device="cuda", generator=g) < case["empty"]
        s["row_of"] = torch.where(drop, -1, order).contiguous()
        s["w"] = torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1) if case["weights"] else None
        if op == "combine":
            s["y"] = torch.empty(T, H, dtype=TORCH[dtype], device="cuda")
        else:
            s["dy"] = _randn(g, (T, H), dtype)
            s["drows"] = torch.zeros(T * k, H, dtype=TORCH[dtype], device="cuda")
            s["dw"] = torch.empty(T, k, device="cuda")
    elif op == "matmul":
        M, N, K, G, way = (case[n] for n in ("M", "N", "K", "G", "way"))
        if way != "dx":
            s["x"] = _randn(g, (M, K), "bf16")
        if way != "y":
            s["dy"] = _randn(g, (M, N), "bf16")
        if way != "dw":
            s["w"] = _randn(g, (G, N, K), "bf16", 0.02)
        s["offsets"] = None
        if G > 1:
            n = torch.tensor(_sizes(case), device="cuda")
            n = n[torch.randperm(G, device="cuda", generator=g)]
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        shape = {"y": (M, N), "dx": (M, K), "dw": (G, N, K)}[way]
        s["out"] = torch.zeros(shape, dtype=TORCH[case["out"]], device="cuda")
        s["add"] = _randn(g, shape, case["out"]) if case["add"] else None
    elif op in ("swiglu", "swiglu_grad"):
        R, I, dtype = case["R"], case["I"], case["dtype"]
        s["gate"], s["up"] = _randn(g, (R, I), dtype, 2.0), _randn(g, (R, I), dtype, 2.0)
        s["used"] = torch.tensor([R - case["tail"]], dtype=torch.int32, device="cuda")
        s["h"] = torch.zeros(R, I, dtype=TORCH[dtype], device="cuda")
        s["codes"] = s["scales"] = None
        if op == "swiglu":
            if case["keep"]:
                s["codes"] = torch.zeros(R, 2 * _padded(I), dtype=F8, device="cuda")
                s["scales"] = torch.zeros(R, 2 * _padded(I) // BLOCK, device="cuda")
        else:
            s["dh"] = _randn(g, (R, I), dtype)
            if case["keep"]:
                parts = [_quant(s[n].float()) for n in ("gate", "up")]
                s["codes"], s["scales"] = (torch.cat(p, 1) for p in zip(*parts))
                s["gate"] = s["up"] = None
            s["dgate"], s["dup"] = torch.zeros_like(s["h"]), torch.zeros_like(s["h"])
    else:
        T, E, k = case["T"], case["E"], case["k"]
        l = torch.randn(T, E, device="cuda", generator=g)
        s["logits"] = l.to(TORCH[case["logits"]])
        s["idx"] = s["logits"].double().sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
        s["dw"] = torch.randn(T, k, device="cuda", generator=g)
        s["dscore"] = torch.rand(E, device="cuda", generator=g) if case["balance"] else None
        s["dlogits"] = torch.empty(T, E, dtype=TORCH[case["logits"]], device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps: the call's sizes and a workspace."""
    import routed_expert_ffn_moe_amd as moe
    case, op = s["case"], s["op"]
    if op == "dispatch":
        s["call"] = moe.make_dispatch(case["T"], case["H"], case["E"], case["k"], x=case["x"])
        s["ws"] = torch.empty(moe.moe_dispatch_workspace_bytes(s["call"]), dtype=torch.uint8, device="cuda")
    elif op in ("combine", "combine_grad"):
        s["call"] = moe.make_combine(case["T"], case["H"], case["k"], case["T"] * case["k"], dtype=case["dtype"])
    elif op == "matmul":
        s["call"] = moe.make_matmul_bf16(case["M"], case["N"], case["K"], G=case["G"], out=case["out"])
    elif op in ("swiglu", "swiglu_grad"):
        s["call"] = moe.make_swiglu(case["R"], case["I"], dtype=case["dtype"])
    else:
        s["call"] = moe.make_select(case["T"], case["E"], case["k"], score=case["score"], renorm=case["renorm"],
                                    scale=case["scale"], logits=case["logits"])


# ---- one pass ---------------------------------------------------------------

def run(s):
    (_run_own if own else _PLAIN[s["op"]])(s)
    return {n: s[n] for n in _OUTPUTS[s["op"]] if s[n] is not None}


_OUTPUTS = {"dispatch": ("rows", "offsets", "row_src", "row_of"), "combine": ("y",), "combine_grad": ("drows", "dw"),
            "matmul": ("out",), "swiglu": ("h", "codes", "scales"), "swiglu_grad": ("dgate", "dup", "h"),
            "select_grad": ("dlogits",)}


def _run_own(s):
    import routed_expert_ffn_moe_amd as moe
    op, call = s["op"], s["call"]
    if op == "dispatch":
        moe.moe_dispatch(call, s["idx"], s["x"], s["sx"], s["rows"], s["offsets"], s["row_src"], s["row_of"], s["ws"])
    elif op == "combine":
        moe.moe_combine(call, s["rows"], s["row_of"], s["w"], s["y"])
    elif op == "combine_grad":
        moe.moe_combine_grad(call, s["dy"], s["rows"], s["row_of"], s["w"], s["drows"], s["dw"])
    elif op == "matmul":
        way = s["case"]["way"]
        if way == "y":
            moe.moe_matmul_bf16(call, s["x"], s["w"], s["out"], s["offsets"], s["add"])
        elif way == "dx":
            moe.moe_matmul_bf16_dx(call, s["dy"], s["w"], s["out"], s["offsets"], s["add"])
        else:
            moe.moe_matmul_bf16_dw(call, s["dy"], s["x"], s["out"], s["offsets"], s["add"])
    elif op == "swiglu":
        moe.moe_swiglu(call, s["gate"], s["up"], s["h"], s["codes"], s["scales"], s["used"])
    elif op == "swiglu_grad":
        moe.moe_swiglu_grad(call, s["gate"], s["up"], s["codes"], s["scales"], s["dh"], s["dgate"], s["dup"], s["h"],
                            s["used"])
    else:
        moe.moe_select_grad(call, s["logits"], s["idx"], s["dw"], s["dscore"], s["dlogits"])


def _rows(codes, scales, width):
    """The values of codes with one scale for each 1 x 128 block."""
    R, Kp = codes.shape
    return (codes.float().view(R, Kp // BLOCK, BLOCK) * scales[:, :, None]).view(R, Kp)[:, :width]


def _dispatch(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    e = s["idx"].flatten().long()
    e = torch.where((e >= 0) & (e < E), e, E)
    order = e.sort(stable=True).indices
    ends = torch.bincount(e, minlength=E + 1)[:E].cumsum(0)
    n = int(ends[-1])
    s["offsets"][1:] = ends
    s["row_src"][:n] = order[:n]
    s["row_of"].fill_(-1)
    s["row_of"].view(-1)[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    x = s["x"] if s["sx"] is None else _rows(s["x"], s["sx"], c["H"]).to(s["rows"].dtype)
    s["rows"][:n] = x[order[:n] // k]


def _combine(s):
    at = s["row_of"].long()
    f = (at >= 0).float() if s["w"] is None else torch.where(at >= 0, s["w"], 0.0)
    acc = torch.zeros(s["y"].shape, device="cuda")
    for j in range(at.shape[1]):
        acc += f[:, j:j + 1] * s["rows"][at[:, j].clamp(min=0)].float()
    s["y"].copy_(acc)


def _combine_grad(s):
    at = s["row_of"].long()
    f = (at >= 0).float() if s["w"] is None else torch.where(at >= 0, s["w"], 0.0)
    dy = s["dy"].float()
    for j in range(at.shape[1]):
        there = (at[:, j] >= 0).nonzero().flatten()
        r = at[there, j]
        s["drows"][r] = (f[there, j:j + 1] * dy[there]).to(s["drows"].dtype)
        s["dw"][:, j] = 0.0
        s["dw"][there, j] = (dy[there] * s["rows"][r].float()).sum(1)


def _matmul(s):
    c = s["case"]
    way, out = c["way"], s["out"]
    ends = [0, c["M"]] if s["offsets"] is None else s["offsets"].tolist()
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        at = i if way == "dw" else slice(lo, hi)
        if way == "y":
            v = s["x"][lo:hi].float() @ s["w"][i].float().t()
        elif way == "dx":
            v = s["dy"][lo:hi].float() @ s["w"][i].float()
        else:
            v = s["dy"][lo:hi].float().t() @ s["x"][lo:hi].float()
        if s["add"] is not None:
            v = v + s["add"][at].float()
        out[at] = v.to(out.dtype)


def _swiglu(s):
    n = s["case"]["R"] - s["case"]["tail"]
    gate, up = s["gate"][:n].float(), s["up"][:n].float()
    s["h"][:n] = (gate / (1.0 + torch.exp(-gate)) * up).to(s["h"].dtype)
    if s["codes"] is not None:
        parts = [_quant(v) for v in (gate, up)]
        s["codes"][:n], s["scales"][:n] = (torch.cat(p, 1) for p in zip(*parts))


def _swiglu_grad(s):
    I, n = s["case"]["I"], s["case"]["R"] - s["case"]["tail"]
    if s["codes"] is None:
        gate, up = s["gate"][:n].float(), s["up"][:n].float()
    else:
        w, b = _padded(I), _padded(I) // BLOCK
        gate = _rows(s["codes"][:n, :w], s["scales"][:n, :b], I)
        up = _rows(s["codes"][:n, w:], s["scales"][:n, b:], I)
    dh = s["dh"][:n].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    for name, v in (("dgate", dh * up * sig * (1.0 + gate * (1.0 - sig))), ("dup", dh * silu), ("h", silu * up)):
        s[name][:n] = v.to(s[name].dtype)


def _select_grad(s):
    """In 64 bits: the ratios of small scores, and differences of gradients that are nearly alike."""
    c = s["case"]
    l, dw, idx = s["logits"].double(), s["dw"].double(), s["idx"].long()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    chosen = score.gather(1, idx)
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        p = chosen / total
        d = (dw - (p * dw).sum(1, keepdim=True)) / total
    else:
        d = dw
    ds = torch.zeros_like(score).scatter_add_(1, idx, d * c["scale"])
    if s["dscore"] is not None:
        ds = ds + s["dscore"].double()
    if c["score"] == "sigmoid":
        dl = ds * score * (1.0 - score)
    else:
        dl = score * (ds - (score * ds).sum(1, keepdim=True))
    s["dlogits"].copy_(dl)


_PLAIN = {"dispatch": _dispatch, "combine": _combine, "combine_grad": _combine_grad, "matmul": _matmul,
          "swiglu": _swiglu, "swiglu_grad": _swiglu_grad, "select_grad": _select_grad}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "dispatch":
        T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
        n = T * k * (1.0 - case["empty"])
        read = T * H * SIZE[case["x"]] if case["x"] != "fp8" else T * (_padded(H) + 4 * (_padded(H) // BLOCK))
        out = SIZE["bf16" if case["x"] == "fp8" else case["x"]]
        return {"bytes": int(read + n * H * out + 8 * T * k + 4 * n + 4 * (E + 1)), "flops": T * k}
    if op in ("combine", "combine_grad"):
        T, H, k, size = case["T"], case["H"], case["k"], SIZE[case["dtype"]]
        n = T * k * (1.0 - case["empty"])
        small = 4 * T * k * (2 if case["weights"] else 1)
        if op == "combine":
            return {"bytes": int((n + T) * H * size + small), "flops": int(2 * n * H)}
        return {"bytes": int((2 * n + T) * H * size + small + 4 * T * k), "flops": int(3 * n * H)}
    if op == "matmul":
        M, N, K = case["M"] - case["tail"], case["N"], case["K"]
        sizes = [M] if case["G"] == 1 else _sizes(case)
        used = sum(n > 0 for n in sizes)
        size = SIZE[case["out"]] * (2 if case["add"] else 1)
        there = {"y": 2 * M * K + 2 * used * N * K + size * M * N, "dx": 2 * M * N + 2 * used * N * K + size * M * K,
                 "dw": 2 * M * (N + K) + size * case["G"] * N * K}[case["way"]]
        return {"bytes": there, "flops": 2 * M * N * K}
    if op in ("swiglu", "swiglu_grad"):
        n, I, size = case["R"] - case["tail"], case["I"], SIZE[case["dtype"]]
        kept = 2 * (_padded(I) + 4 * (_padded(I) // BLOCK))
        if op == "swiglu":
            return {"bytes": n * (3 * I * size + (kept if case["keep"] else 0)) + 4, "flops": 8 * n * I}
        return {"bytes": n * (4 * I * size + (kept if case["keep"] else 2 * I * size)) + 4, "flops": 14 * n * I}
    T, E, k = case["T"], case["E"], case["k"]
    return {"bytes": T * E * 2 * SIZE[case["logits"]] + 8 * T * k + (4 * E if case["balance"] else 0),
            "flops": 6 * T * E}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    out = {n: s[n].double() if s[n].is_floating_point() else s[n]
           for n in _OUTPUTS[s["op"]] if s[n] is not None}
    _EXACT[s["op"]](s, out)
    return out


def _exact_dispatch(s, out):
    """One expert after the other: its pairs in the order of the tokens."""
    c = s["case"]
    x = s["x"].double()
    if s["sx"] is not None:
        x = (x * s["sx"].double().repeat_interleave(BLOCK, 1))[:, :c["H"]]
    out["row_of"].fill_(-1)
    at = 0
    for e in range(c["E"]):
        pairs = (s["idx"].flatten() == e).nonzero().flatten()
        n = pairs.numel()
        out["offsets"][e + 1] = at + n
        out["row_src"][at:at + n] = pairs.to(torch.int32)
        out["row_of"].view(-1)[pairs] = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        out["rows"][at:at + n] = x[torch.div(pairs, c["k"], rounding_mode="floor")]
        at += n


def _slots(s):
    """(slot's tokens, slots, rows, weights) of the slots in use."""
    t, j = (s["row_of"] >= 0).nonzero(as_tuple=True)
    w = torch.ones(t.numel(), dtype=torch.float64, device="cuda") if s["w"] is None else s["w"][t, j].double()
    return t, j, s["row_of"][t, j].long(), w


def _exact_combine(s, out):
    t, _, r, w = _slots(s)
    out["y"].zero_()
    step = 1 << 14
    for i in range(0, t.numel(), step):
        out["y"].index_add_(0, t[i:i + step], s["rows"][r[i:i + step]].double() * w[i:i + step, None])


def _exact_combine_grad(s, out):
    t, j, r, w = _slots(s)
    out["dw"].zero_()
    step = 1 << 14
    for i in range(0, t.numel(), step):
        a, b = t[i:i + step], r[i:i + step]
        dy = s["dy"][a].double()
        out["drows"][b] = dy * w[i:i + step, None]
        out["dw"][a, j[i:i + step]] = torch.linalg.vecdot(dy, s["rows"][b].double())


def _exact_matmul(s, out):
    way, v = s["case"]["way"], out["out"]
    ends = [0, s["case"]["M"]] if s["offsets"] is None else s["offsets"].tolist()
    for i in range(s["case"]["G"]):
        rows = slice(ends[i], ends[i + 1])
        at = i if way == "dw" else rows
        if way == "dw":
            v[at] = torch.matmul(s["dy"][rows].double().t(), s["x"][rows].double())
        elif way == "dx":
            v[at] = torch.matmul(s["dy"][rows].double(), s["w"][i].double())
        else:
            v[at] = torch.matmul(s["w"][i].double(), s["x"][rows].double().t()).t()
        if s["add"] is not None:
            v[at] += s["add"][at].double()


def _exact_codes(x):
    """(codes, scales) in 64 bits: each value over its block's scale, to the nearest E4M3 value, ties to the even one."""
    R, K = x.shape
    p = torch.nn.functional.pad(x, (0, _padded(K) - K)).view(R, -1, BLOCK)
    top = p.abs().amax(2).clamp(min=TINY)
    v = p * E4M3_MAX / top[:, :, None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)  # subnormal below 2^-6
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX).view(R, -1), top / E4M3_MAX


def _exact_swiglu(s, out):
    n = s["case"]["R"] - s["case"]["tail"]
    gate, up = s["gate"][:n].double(), s["up"][:n].double()
    out["h"][:n] = torch.sigmoid(gate) * gate * up
    if s["codes"] is not None:
        (gc, gs), (uc, us) = _exact_codes(gate), _exact_codes(up)
        out["codes"][:n], out["scales"][:n] = torch.cat([gc, uc], 1), torch.cat([gs, us], 1)


def _exact_swiglu_grad(s, out):
    """The derivatives by differentiation of the definition."""
    I, n = s["case"]["I"], s["case"]["R"] - s["case"]["tail"]
    if s["codes"] is None:
        gate, up = s["gate"][:n].double(), s["up"][:n].double()
    else:
        v = s["codes"][:n].double() * s["scales"][:n].double().repeat_interleave(BLOCK, 1)
        gate, up = v[:, :I], v[:, _padded(I):_padded(I) + I]
    gate, up = gate.contiguous().requires_grad_(), up.contiguous().requires_grad_()
    with torch.enable_grad():
        h = gate * torch.sigmoid(gate) * up
        out["dgate"][:n], out["dup"][:n] = torch.autograd.grad(h, (gate, up), s["dh"][:n].double())
    out["h"][:n] = h.detach()


def _exact_select_grad(s, out):
    """The derivative by differentiation of the weights (and of the balance loss)."""
    c = s["case"]
    l = s["logits"].double().requires_grad_()
    with torch.enable_grad():
        score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
        w = torch.gather(score, 1, s["idx"].long())
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        loss = (w * c["scale"] * s["dw"].double()).sum()
        if s["dscore"] is not None:
            loss = loss + (score * s["dscore"].double()).sum()
        out["dlogits"] = torch.autograd.grad(loss, l)[0]


_EXACT = {"dispatch": _exact_dispatch, "combine": _exact_combine, "combine_grad": _exact_combine_grad,
          "matmul": _exact_matmul, "swiglu": _exact_swiglu, "swiglu_grad": _exact_swiglu_grad,
          "select_grad": _exact_select_grad}
