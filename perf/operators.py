"""Cases of the FP8 and routing operators, measured against their plain forms.

Four operators that a mixture-of-experts layer with 8-bit weights is made of:

``select``   the experts of each token from the router's logits: softmax or
             sigmoid scores, a balancing bias that counts in the selection
             only, expert groups, renormalised and scaled weights
``quant``    rows (or weight matrices) to E4M3 codes with one fp32 scale per
             1 x 128 (128 x 128) block
``matmul``   the product of such codes, scaled block by block along K: one
             matrix, or one per group of rows
``experts``  the routed experts' FFN on E4M3 weights with given routing

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


def listed():
    return [
        # one decoded token: scores of 256 experts, limited to 4 of 8 groups
        dict(name="select-decode-groups", op="select", T=1, E=256, k=8, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_score="top2", renorm=True, scale=2.5, logits="f32"),
        # a prefill chunk routed by softmax over logits kept in bf16 (equal logits occur)
        dict(name="select-chunk-softmax", op="select", T=2048, E=256, k=8, score="softmax", bias=False,
             n_group=1, topk_group=1, group_score="max", renorm=True, scale=1.0, logits="bf16"),
        # a long pass of the wide layer, balanced by a bias
        dict(name="select-long-bias", op="select", T=8192, E=384, k=6, score="sigmoid", bias=True,
             n_group=1, topk_group=1, group_score="max", renorm=True, scale=1.0, logits="f32"),
        # the activations of a prefill chunk
        dict(name="quant-chunk", op="quant", R=2048, K=2048, rows=1, src="bf16"),
        # one expert bank's worth of fp32 weight rows at load time, an odd width
        dict(name="quant-weights", op="quant", R=8192, K=4000, rows=128, src="f32"),
        # a projection of one decoded token
        dict(name="matmul-decode", op="matmul", M=1, N=4096, K=4096, G=1, tail=0, out="bf16"),
        # a short ragged pass, fp32 out
        dict(name="matmul-ragged", op="matmul", M=601, N=2050, K=776, G=1, tail=0, out="f32"),
        # a projection of a long prefill pass: bound by the matrix cores
        dict(name="matmul-long", op="matmul", M=8192, N=4096, K=4096, G=1, tail=0, out="bf16"),
        # the rows of a prefill chunk, eight experts each, grouped by expert; some rows behind the last group
        dict(name="matmul-grouped", op="matmul", M=16384, N=1536, K=2048, G=256, tail=37, out="bf16"),
        # the experts of one decoded token
        dict(name="experts-decode", op="experts", T=1, H=2048, E=256, k=8, I=768, skew=0.0),
        # a prefill chunk with Zipf-skewed routing
        dict(name="experts-chunk-zipf", op="experts", T=2048, H=2048, E=256, k=8, I=768, skew=1.1),
        # the wide layer at a long pass
        dict(name="experts-wide-long", op="experts", T=8192, H=4096, E=384, k=6, I=2048, skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "quant", "matmul", "matmul", "experts", "experts"])
    if op == "select":
        ng = rng.choice([1, 1, 4, 8])
        per = rng.randint(4, 64)
        E = ng * per
        tg = 1 if ng == 1 else rng.randint(1, ng)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(10, tg * per if ng > 1 else E)),
                    score=score, bias=rng.random() < 0.6, n_group=ng, topk_group=tg,
                    group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.8,
                    scale=rng.choice([1.0, 2.5]), logits=rng.choice(["f32", "bf16"]))
    if op == "quant":
        return dict(op=op, R=_log(rng, 1, 8192), K=_log(rng, 64, 8192), rows=rng.choice([1, 128]),
                    src=rng.choice(["f32", "bf16"]))
    if op == "matmul":
        out = rng.choice(["f32", "bf16"])
        if rng.random() < 0.6:
            return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 48, 4096), K=_log(rng, 64, 4096),
                        G=1, tail=0, out=out)
        M = _log(rng, 2, 16384)
        return dict(op=op, M=M, N=128 * rng.randint(1, 12), K=128 * rng.randint(1, 16),
                    G=_log(rng, 2, 256), tail=rng.randint(0, max(0, M // 50)), out=out)
    E = rng.choice([8, 16, 64, 128, 256])
    return dict(op=op, T=_log(rng, 1, 4096), H=128 * rng.randint(2, 32), E=E, k=rng.randint(1, min(8, E)),
                I=128 * rng.randint(1, 16), skew=rng.choice([0.0, 0.0, 1.1]))


# ---- inputs ---------------------------------------------------------------

def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _codes(g, rows, width, sigma, out=None):
    """E4M3 codes of normal draws whose largest reach the format's end."""
    out = torch.empty(rows, width, dtype=F8, device="cuda") if out is None else out
    step = max(1, (1 << 28) // width)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        v = torch.empty(n, width, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma, generator=g)
        out[r:r + n] = v.clamp_(-E4M3_MAX, E4M3_MAX).to(F8)
    return out


def _scales(g, shape, size):
    return torch.rand(shape, device="cuda", generator=g).mul_(1.0).add_(0.5).mul_(size)


def _sizes(case):
    """Rows of each group, largest first: Zipf shares of all rows but the tail (some groups get none)."""
    M, G = case["M"] - case["tail"], case["G"]
    share = [1.0 / (i + 1) for i in range(G)]
    s = sum(share)
    n = [int(M * v / s) for v in share]
    n[0] += M - sum(n)
    return n


def _touched(case):
    """Experts that get a row, on average."""
    T, E, k, skew = case["T"], case["E"], case["k"], case["skew"]
    p = [(i + 1) ** -skew for i in range(E)]
    s = sum(p)
    return min(E, sum(1.0 - (1.0 - min(1.0, k * v / s)) ** T for v in p))


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, op=op)
    if op == "select":
        T, E = case["T"], case["E"]
        s["logits"] = torch.randn(T, E, device="cuda", generator=g).to(TORCH[case["logits"]])
        s["bias"] = torch.randn(E, device="cuda", generator=g) * 0.1 if case["bias"] else None
        s["idx"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, case["k"], dtype=torch.float32, device="cuda")
    elif op == "quant":
        R, K = case["R"], case["K"]
        x = torch.randn(R, K, device="cuda", generator=g)
        if case["rows"] == 128:
            x *= 0.02
        else:  # activations: a few channels carry large values
            x *= torch.exp(torch.randn(1, K, device="cuda", generator=g))
        s["x"] = x.to(TORCH[case["src"]])
        s["codes"] = torch.empty(R, _padded(K), dtype=F8, device="cuda")
        s["scales"] = torch.empty(-(-R // case["rows"]), _padded(K) // BLOCK, device="cuda")
    elif op == "matmul":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        Kp = _padded(K)
        s["a"] = _codes(g, M, Kp, 150.0)
        s["b"] = _codes(g, G * N, Kp, 112.0).view(G, N, Kp)
        if Kp > K:
            s["a"][:, K:] = 0
            s["b"][:, :, K:] = 0
        s["sa"] = _scales(g, (M, Kp // BLOCK), 1.0 / 150)
        s["sb"] = _scales(g, (G, _padded(N) // BLOCK, Kp // BLOCK), 0.02 / 112)
        s["offsets"] = None
        if G > 1:
            n = torch.tensor(_sizes(case), device="cuda")
            n = n[torch.randperm(G, device="cuda", generator=g)]
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        s["y"] = torch.zeros(M, N, dtype=TORCH[case["out"]], device="cuda")
    else:
        T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
        s["x"] = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
        for name, n, d in (("gate", I, H), ("up", I, H), ("down", H, I)):
            s["w_" + name] = _codes(g, E * n, d, 112.0).view(E, n, d)
            s["s_" + name] = _scales(g, (E, n // BLOCK, d // BLOCK), 0.02 / 112)
        # distinct experts per token, drawn by their Zipf shares (uniform without a skew)
        lean = -case["skew"] * torch.log(1.0 + torch.randperm(E, device="cuda", generator=g))
        u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-9, 1 - 1e-7)
        z, idx = (lean - torch.log(-torch.log(u))).topk(k, dim=1)
        s["idx"] = idx.to(torch.int32).contiguous()
        s["w"] = torch.softmax(z, dim=1).contiguous()
        s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps: the call's sizes, its weights' struct and a workspace."""
    import routed_expert_ffn_moe_amd as moe
    case, op = s["case"], s["op"]
    if op == "select":
        s["call"] = moe.make_select(case["T"], case["E"], case["k"], score=case["score"],
                                    n_group=case["n_group"], topk_group=case["topk_group"],
                                    group_score=case["group_score"], renorm=case["renorm"],
                                    scale=case["scale"], logits=case["logits"])
    elif op == "quant":
        s["call"] = moe.make_quant(case["R"], case["K"], src=case["src"], block_rows=case["rows"])
    elif op == "matmul":
        s["call"] = moe.make_matmul(case["M"], case["N"], case["K"], G=case["G"], out=case["out"])
    else:
        s["call"] = moe.make_shape(case["T"], case["H"], case["E"], case["k"], case["I"],
                                   act="bf16", w="fp8")
        s["weights"] = moe.make_weights(None, s["w_gate"], s["w_up"], s["w_down"], s_gate=s["s_gate"],
                                        s_up=s["s_up"], s_down=s["s_down"])
        s["ws"] = torch.empty(moe.moe_workspace_bytes(s["call"]), dtype=torch.uint8, device="cuda")


# ---- one pass ---------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        import routed_expert_ffn_moe_amd as moe
        if op == "select":
            moe.moe_select(s["call"], s["logits"], s["bias"], s["idx"], s["w"])
            return {"idx": s["idx"], "w": s["w"]}
        if op == "quant":
            moe.moe_quant_fp8(s["call"], s["x"], s["codes"], s["scales"])
            return {"codes": s["codes"], "scales": s["scales"]}
        if op == "matmul":
            moe.moe_matmul_fp8(s["call"], s["a"], s["sa"], s["b"], s["sb"], s["y"], s["offsets"])
            return {"y": s["y"]}
        moe.moe_experts(s["call"], s["weights"], s["x"], s["idx"], s["w"], s["y"], s["ws"])
        return {"y": s["y"]}
    if op == "select":
        return _select(s)
    if op == "quant":
        codes, scales = _quant(s["x"].float(), s["case"]["rows"])
        s["codes"].copy_(codes.to(F8))
        s["scales"].copy_(scales)
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "matmul":
        return _matmul(s)
    return _experts(s)


def _select(s):
    """Scores in 64 bits: the order of near-equal ones decides which experts run."""
    c = s["case"]
    T, E, k, ng = c["T"], c["E"], c["k"], c["n_group"]
    l = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"].double()
    if ng > 1:
        top = key.view(T, ng, E // ng).sort(dim=2, descending=True).values
        value = top[:, :, 0] if c["group_score"] == "max" else top[:, :, :2].sum(2)
        rank = value.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros(T, ng, dtype=torch.bool, device="cuda").scatter_(1, rank, True)
        key = torch.where(keep.repeat_interleave(E // ng, 1), key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    s["idx"].copy_(idx)
    s["w"].copy_(w * c["scale"])
    return {"idx": s["idx"], "w": s["w"]}


def _quant(x, rows):
    """(codes as fp32, scales) of fp32 rows: one scale for each `rows` x 128 block.  Products by 448 before the
    division: the quotient of two bf16 values that lies half way between two codes then stays half way."""
    R, K = x.shape
    Rp, Kp = -(-R // rows) * rows, _padded(K)
    p = torch.zeros(Rp, Kp, device=x.device)
    p[:R, :K] = x
    p = p.view(Rp // rows, rows, Kp // BLOCK, BLOCK)
    top = p.abs().amax((1, 3)).clamp(min=TINY)
    return (p * E4M3_MAX / top[:, None, :, None]).to(F8).float().view(Rp, Kp)[:R], top / E4M3_MAX


def _rows(codes, scales):
    """The values of codes with one scale for each 1 x 128 block."""
    R, Kp = codes.shape
    return (codes.float().view(R, Kp // BLOCK, BLOCK) * scales[:, :, None]).view(R, Kp)


def _matrix(codes, scales):
    """The values of a matrix of codes with one scale for each 128 x 128 block."""
    N, Kp = codes.shape
    if N % BLOCK:
        return codes.float() * scales.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)
    return (codes.float().view(N // BLOCK, BLOCK, Kp // BLOCK, BLOCK) * scales[:, None, :, None]).view(N, Kp)


def _matmul(s):
    a = _rows(s["a"], s["sa"])
    if s["offsets"] is None:
        s["y"].copy_(a @ _matrix(s["b"][0], s["sb"][0]).t())
        return {"y": s["y"]}
    off = s["offsets"].tolist()
    for i in range(s["case"]["G"]):
        if off[i + 1] > off[i]:
            s["y"][off[i]:off[i + 1]] = (a[off[i]:off[i + 1]] @ _matrix(s["b"][i], s["sb"][i]).t()).to(s["y"].dtype)
    return {"y": s["y"]}


def _experts(s):
    c = s["case"]
    k = c["k"]
    x = _rows(*_quant(s["x"].float(), 1))
    pair_e, pair = s["idx"].flatten().long().sort(stable=True)
    off = torch.cat([pair_e.new_zeros(1), torch.bincount(pair_e, minlength=c["E"]).cumsum(0)]).tolist()
    out = torch.empty(c["T"] * k, c["H"], device="cuda")
    for e in range(c["E"]):
        if off[e + 1] == off[e]:
            continue
        rows = pair[off[e]:off[e + 1]]
        xe = x[rows // k]
        gate = xe @ _matrix(s["w_gate"][e], s["s_gate"][e]).t()
        up = xe @ _matrix(s["w_up"][e], s["s_up"][e]).t()
        h = _rows(*_quant(gate / (1.0 + torch.exp(-gate)) * up, 1))
        out[rows] = h @ _matrix(s["w_down"][e], s["s_down"][e]).t()
    s["y"].copy_((out.view(c["T"], k, -1) * s["w"][:, :, None]).sum(1))
    return {"y": s["y"]}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["logits"] == "f32" else 2) + (4 * E if case["bias"] else 0) + 8 * T * k,
                "flops": 4 * T * E}
    if op == "quant":
        R, K = case["R"], case["K"]
        return {"bytes": R * K * (4 if case["src"] == "f32" else 2) + R * _padded(K) + 4 * -(-R // case["rows"]) * (_padded(K) // BLOCK),
                "flops": 2 * R * K}
    if op == "matmul":
        M, N, K = case["M"] - case["tail"], case["N"], _padded(case["K"])
        G = 1 if case["G"] == 1 else sum(n > 0 for n in _sizes(case))
        return {"bytes": M * K + 4 * M * K // BLOCK + G * (N * K + 4 * (_padded(N) // BLOCK) * (K // BLOCK))
                + M * N * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    T, H, k, I = (case[n] for n in ("T", "H", "k", "I"))
    return {"bytes": int(_touched(case) * 3 * H * I * (1 + 4 / BLOCK ** 2)) + 4 * T * H + 8 * T * k,
            "flops": 6 * T * k * H * I}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "select":
        return _exact_select(s)
    if op == "quant":
        codes, scales = _exact_quant(s["x"].double(), case["rows"])
        return {"codes": codes, "scales": scales}
    if op == "matmul":
        a = s["a"].double() * s["sa"].double().repeat_interleave(BLOCK, 1)
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        ends = [0, case["M"]] if s["offsets"] is None else s["offsets"].tolist()
        for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                y[lo:hi] = a[lo:hi] @ _exact_matrix(s["b"][i], s["sb"][i]).t()
        return {"y": y}
    codes, scales = _exact_quant(s["x"].double(), 1)
    x = codes * scales.repeat_interleave(BLOCK, 1)
    y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        gate, up = (x[t] @ _exact_matrix(s["w_" + n][e], s["s_" + n][e]).t() for n in ("gate", "up"))
        codes, scales = _exact_quant(gate * torch.sigmoid(gate) * up, 1)
        o = (codes * scales.repeat_interleave(BLOCK, 1)) @ _exact_matrix(s["w_down"][e], s["s_down"][e]).t()
        y.index_add_(0, t, o * s["w"][t, j].double()[:, None])
    return {"y": y}


def _exact_select(s):
    """The definition by repeated choice: the best group, then the best expert, one at a time."""
    c = s["case"]
    T, E, ng = c["T"], c["E"], c["n_group"]
    l = s["logits"].double()
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    key = score.clone() if s["bias"] is None else score + s["bias"].double()
    rows = torch.arange(T, device="cuda")
    if ng > 1:
        groups = key.view(T, ng, E // ng)
        value = groups.amax(2)
        if c["group_score"] == "top2":
            value = groups.topk(min(2, E // ng), dim=2).values.sum(2)
        open_ = torch.zeros(T, ng, dtype=torch.bool, device="cuda")
        for _ in range(c["topk_group"]):
            first = (value == value.amax(1, keepdim=True)).to(torch.int8).argmax(1)
            open_[rows, first] = True
            value[rows, first] = -math.inf
        key = key.masked_fill(~open_[:, :, None].expand(T, ng, E // ng).reshape(T, E), -math.inf)
    idx, w = [], []
    for _ in range(c["k"]):
        first = (key == key.amax(1, keepdim=True)).to(torch.int8).argmax(1)
        idx.append(first)
        w.append(score[rows, first])
        key[rows, first] = -math.inf
    idx, w = torch.stack(idx, 1).to(torch.int32), torch.stack(w, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx, "w": w * c["scale"]}


def _exact_quant(x, rows):
    """(codes, scales) in 64 bits: each value over its block's scale, to the nearest E4M3 value, ties to the even one."""
    R, K = x.shape
    Rp, Kp = -(-R // rows) * rows, _padded(K)
    p = torch.nn.functional.pad(x, (0, Kp - K, 0, Rp - R)).view(Rp // rows, rows, Kp // BLOCK, BLOCK)
    top = p.abs().amax((1, 3)).clamp(min=TINY)
    v = p * E4M3_MAX / top[:, None, :, None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)  # subnormal below 2^-6
    v = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return v.view(Rp, Kp)[:R], top / E4M3_MAX


def _exact_matrix(codes, scales):
    N, Kp = codes.shape
    s = scales.double()[:, None, :, None].expand(-1, BLOCK, -1, BLOCK).reshape(-1, Kp)
    return codes.double() * s[:N]
