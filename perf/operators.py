"""Rotary positions, attention over packed prompts (with its gradients) and attention of drafted token trees
over a cache: the cases that are timed, and the operators in plain torch.

    own = False    run() computes the plain form (elementary torch operations in fp32)
    own = True     run() makes the calls a user makes of hierarchical_block_sparse_pyr_b200
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ELT = {"bf16": 2, "f32": 4}


# ---- cases -------------------------------------------------------------------------------------------------

def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


def listed():
    return [
        # one decode step of the 32-sequence workload: the new token of every sequence, far into its context
        dict(name="rope_decode", op="rope", B=32, Hq=32, Hkv=8, N=1, d=128, rot=128, dtype="bf16", layout="half",
             scaling="none", inverse=False, where="given", first=131071, order="hnd"),
        # the queries and keys of a 32K prompt, 16 heads, stretched from a shorter training length
        dict(name="rope_prompt_32k", op="rope", B=1, Hq=16, Hkv=16, N=32768, d=128, rot=128, dtype="bf16",
             layout="half", scaling="yarn", inverse=False, where="offset", first=0, order="hnd"),
        # gradient of a rotation of half of each head, adjacent pairs, single precision, an odd length
        dict(name="rope_partial_f32_grad", op="rope", B=2, Hq=32, Hkv=8, N=4097, d=64, rot=32, dtype="f32",
             layout="interleaved", scaling="linear", inverse=True, where="given", first=0, order="nhd"),
        # a few short prompts arriving together: latency counts
        dict(name="prompt_short", op="prompt", lens="1,37,64,130", pad=0, Hq=8, Hkv=2, d=128, dtype="bf16",
             order="nhd"),
        # a serving batch of ragged prompts, grouped heads, token-major activations
        dict(name="prompt_ragged_gqa", op="prompt", lens="4096,1,777,2500,63,1025,129,3000,512,1900,300,640,1441",
             pad=17, Hq=32, Hkv=8, d=128, dtype="bf16", order="nhd"),
        # one long document packed with shorter ones, 16 heads, 32K tokens in all
        dict(name="prompt_long_mha", op="prompt", lens="24001,6000,2500,267", pad=0, Hq=16, Hkv=16, d=128,
             dtype="bf16", order="hnd"),
        # gradients at the size of the single-precision workload: 2 heads of 64, 4K tokens
        dict(name="prompt_grad_f32", op="prompt_grad", lens="2047,1,1500,548", pad=0, Hq=2, Hkv=2, d=64, dtype="f32",
             order="hnd"),
        # a training batch of ragged documents, grouped heads
        dict(name="prompt_grad_ragged_gqa", op="prompt_grad", lens="2048,1,777,1500,63,1025,129,1700,512,437", pad=0,
             Hq=32, Hkv=8, d=128, dtype="bf16", order="nhd"),
        # a training batch with one long document, 16 heads, 32K tokens in all
        dict(name="prompt_grad_long_mha", op="prompt_grad", lens="24001,6000,2500,267", pad=0, Hq=16, Hkv=16, d=128,
             dtype="bf16", order="hnd"),
        # one conversation with a short chain of drafts: latency counts
        dict(name="tree_small", op="tree", lens="1000", slack=24, T=8, Hq=32, Hkv=8, d=128, dtype="bf16",
             shape="chain", order="hnd"),
        # wide trees over middling contexts
        dict(name="tree_wide", op="tree", lens="32000,511,7777,15000", slack=704, T=64, Hq=32, Hkv=8, d=128,
             dtype="bf16", shape="random", order="nhd"),
        # the 32-sequence decode workload with ragged contexts up to 128K and trees of 16
        dict(name="tree_serving_128k", op="tree",
             lens="131056,1,64,1000,2047,4096,5000,7777,9001,12000,16384,20000,23456,30000,33333,40000,"
                  "45000,50001,55555,60000,65536,70000,75000,80000,88888,90000,95000,100000,111111,120000,125000,130000",
             slack=0, T=16, Hq=32, Hkv=8, d=128, dtype="bf16", shape="random", order="hnd"),
    ]


_HEADS = [(2, 2), (4, 2), (8, 1), (8, 2), (8, 8), (16, 16), (32, 8)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, total, parts):
    """`parts` lengths of at least 1 that add up to total, spread over orders of magnitude."""
    w = [math.exp(rng.uniform(0.0, 4.0)) for _ in range(parts)]
    rest = total - parts
    out = [1 + int(rest * x / sum(w)) for x in w]
    out[rng.randrange(parts)] += total - sum(out)
    return out


def _pairs(lens):
    return sum(n * (n + 1) // 2 for n in lens)


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "prompt_grad", "prompt_grad", "tree", "tree"])
    order = rng.choice(["hnd", "nhd"])
    if op == "rope":
        Hq, Hkv = rng.choice(_HEADS)
        d = rng.choice([64, 128])
        dtype = rng.choice(["bf16", "f32"])
        B = _log_int(rng, 1, 32)
        most = 32768 * 32 * 128 * 2 // (B * (Hq + Hkv) * d * _ELT[dtype])
        N = _log_int(rng, 1, min(32768, most))
        rot = rng.choice([d, d, d // 2, d // 4])
        return dict(op="rope", B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, rot=rot, dtype=dtype,
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    inverse=rng.random() < 0.5, where=rng.choice(["given", "offset"]), first=_log_int(rng, 1, 1000000),
                    order=order)
    if op == "tree":
        Hq, Hkv = rng.choice(_HEADS)
        d = rng.choice([64, 128])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        B = _log_int(rng, 1, 32)
        longest = 131056 if dtype == "bf16" else 16384
        lens = [_log_int(rng, 1, longest) for _ in range(B)]
        return dict(op="tree", lens=_text(lens), slack=rng.randrange(0, 200), T=_log_int(rng, 1, 64), Hq=Hq, Hkv=Hkv,
                    d=d, dtype=dtype, shape=rng.choice(["chain", "random"]), order=order)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hq, Hkv = rng.choice(_HEADS)
    limit = _pairs([24001, 6000, 2500, 267]) * 16 if dtype == "bf16" else _pairs([2048, 2048]) * 16
    while True:
        T = _log_int(rng, 1, 32768 if dtype == "bf16" else 4096)
        S = _log_int(rng, 1, min(64, T))
        lens = _split(rng, T, S)
        if _pairs(lens) * Hq <= limit and max(lens) <= 24001:
            break
    return dict(op=op, lens=_text(lens), pad=rng.choice([0, 0, 5, 100]), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, order=order)


def work(case):
    e = _ELT[case["dtype"]]
    d = case["d"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        n = case["B"] * case["N"]
        return {"bytes": 2 * n * (Hq + Hkv) * d * e + (4 * n if case["where"] == "given" else 0),
                "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    lens = _ints(case["lens"])
    if case["op"] == "tree":
        T = case["T"]
        return {"bytes": sum(n + T for n in lens) * 2 * Hkv * d * e + len(lens) * T * Hq * (2 * d * e + 4),
                "flops": 4 * d * Hq * T * sum(n + 1 for n in lens)}
    T = sum(lens)
    if case["op"] == "prompt":
        return {"bytes": T * (2 * Hq + 2 * Hkv) * d * e + 4 * T * Hq, "flops": 4 * d * Hq * _pairs(lens)}
    return {"bytes": T * (4 * Hq + 4 * Hkv) * d * e + 4 * T * Hq, "flops": 10 * d * Hq * _pairs(lens)}


# ---- inputs ------------------------------------------------------------------------------------------------

def _empty(order, B, H, N, d, dtype):
    """A [B, H, N, d] tensor whose memory is head-major ("hnd") or token-major ("nhd")."""
    if order == "hnd":
        return torch.empty((B, H, N, d), dtype=dtype, device="cuda")
    return torch.empty((B, N, H, d), dtype=dtype, device="cuda").transpose(1, 2)


def _normal(gen, order, B, H, N, d, dtype, offsets=False):
    """N(0, 1) values; with offsets, every 64 rows of a head share an offset vector N(0, 0.5^2), as the
    keys of the framework's own workloads do."""
    x = _empty(order, B, H, N, d, dtype)
    for b in range(B):
        y = torch.randn((H, N, d), generator=gen, device="cuda", dtype=torch.float32)
        if offsets:
            o = torch.randn((H, (N + 63) // 64, 1, d), generator=gen, device="cuda", dtype=torch.float32)
            y += 0.5 * o.expand(-1, -1, 64, -1).reshape(H, -1, d)[:, :N]
        x[b].copy_(y)
    return x


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


_BASE = 10000.0
_TRAINED = 8192  # length that the scaled rotations stretch


def _frequencies(case):
    """(angle per position of every pair, factor on the result), in Python's doubles."""
    n = case["rot"] // 2
    rot, kind, factor = case["rot"], case["scaling"], 4.0
    f = [_BASE ** (-2.0 * i / rot) for i in range(n)]
    if kind == "linear":
        return [x / factor for x in f], 1.0
    if kind == "ntk":
        base = _BASE * factor ** (rot / (rot - 2.0))
        return [base ** (-2.0 * i / rot) for i in range(n)], 1.0
    if kind == "yarn":
        # turns over the trained length: pairs above 32 keep their speed, pairs below 1 are slowed by
        # the factor, a linear ramp over the pair index joins them
        at = lambda turns: rot * math.log(_TRAINED / (turns * 2 * math.pi)) / (2 * math.log(_BASE))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(n)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _parents(case, gen):
    B, T = len(_ints(case["lens"])), case["T"]
    if case["shape"] == "chain":
        return torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    u = torch.rand((B, T), generator=gen, device="cuda", dtype=torch.float64)
    t = torch.arange(T, device="cuda", dtype=torch.float64)
    return (torch.floor(u * (t + 1)) - 1).clamp_(max=t - 1).to(torch.int32)  # uniform in -1 .. t - 1


def prepare(case, seed):
    gen = _generator(seed)
    dt = _DT[case["dtype"]]
    Hq, Hkv, d, order = case["Hq"], case["Hkv"], case["d"], case["order"]
    st = {"case": case}
    if own:
        import hierarchical_block_sparse_pyr_b200 as P
        st["P"] = P
    if case["op"] == "rope":
        B, N = case["B"], case["N"]
        st["Q"] = _normal(gen, order, B, Hq, N, d, dt)
        st["K"] = _normal(gen, order, B, Hkv, N, d, dt)
        st["Qo"], st["Ko"] = _empty(order, B, Hq, N, d, dt), _empty(order, B, Hkv, N, d, dt)
        st["pos"] = None
        if case["where"] == "given":
            st["pos"] = torch.randint(max(case["first"] - 100, 0), case["first"] + 4 * N, (B, N), generator=gen,
                                      device="cuda", dtype=torch.int32)
        st["freq"] = _frequencies(case)
        if own:
            kw = {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=4.0),
                  "yarn": dict(scaling="yarn", factor=4.0, trained=_TRAINED)}[case["scaling"]]
            st["spec"] = P.rope_spec(d, case["rot"], base=_BASE, layout=case["layout"], **kw)
        return st
    lens = _ints(case["lens"])
    if case["op"] == "tree":
        B, T = len(lens), case["T"]
        N = max(lens) + T + case["slack"]
        st["Q"] = _normal(gen, order, B, Hq, T, d, dt)
        st["K"] = _normal(gen, order, B, Hkv, N, d, dt, offsets=True)
        st["V"] = _normal(gen, order, B, Hkv, N, d, dt)
        st["lens_host"] = lens
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["parent"] = _parents(case, gen)
        st["O"] = _empty(order, B, Hq, T, d, dt)
        st["lse"] = torch.empty((B, Hq, T), dtype=torch.float32, device="cuda")
        if own:
            st["shape"] = P.tree_shape(B, Hq, Hkv, N, T, d, dt)
            st["workspace"] = torch.empty(P.tree_workspace_bytes(st["shape"]), dtype=torch.uint8, device="cuda")
        return st
    T = sum(lens) + case["pad"]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st["cu_host"] = cu
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["Q"] = _normal(gen, order, 1, Hq, T, d, dt)[0]
    st["K"] = _normal(gen, order, 1, Hkv, T, d, dt, offsets=True)[0]
    st["V"] = _normal(gen, order, 1, Hkv, T, d, dt)[0]
    # rows behind the last sequence belong to the caller and keep what they held
    st["O"] = _empty(order, 1, Hq, T, d, dt)[0].zero_()
    st["lse"] = torch.zeros((Hq, T), dtype=torch.float32, device="cuda")
    if own:
        st["shape"] = P.packed_shape(len(lens), T, Hq, Hkv, d, dt)
        st["plan"] = P.packed_plan(st["shape"], st["cu"])
    if case["op"] == "prompt_grad":
        st["dO"] = _normal(gen, order, 1, Hq, T, d, dt)[0]
        _plain_prompt(st)  # what the forward pass left: O and lse
        st["dQ"] = _empty(order, 1, Hq, T, d, dt)[0].zero_()
        st["dK"] = _empty(order, 1, Hkv, T, d, dt)[0].zero_()
        st["dV"] = _empty(order, 1, Hkv, T, d, dt)[0].zero_()
        if own:
            st["delta"] = torch.empty((Hq, T), dtype=torch.float32, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if not own:
        return {"rope": _plain_rope, "prompt": _plain_prompt, "prompt_grad": _plain_prompt_grad,
                "tree": _plain_tree}[case["op"]](state)
    P = state["P"]
    if case["op"] == "rope":
        P.rope_apply(state["spec"], state["Q"], state["K"], state["Qo"], state["Ko"], pos=state["pos"],
                     pos_offset=case["first"] if state["pos"] is None else 0, inverse=case["inverse"])
        return {"Q": state["Qo"], "K": state["Ko"]}
    if case["op"] == "tree":
        P.tree_forward(state["shape"], state["Q"], state["K"], state["V"], state["lens"], state["parent"], state["O"],
                       state["lse"], workspace=state["workspace"])
        return {"O": state["O"], "lse": state["lse"]}
    if case["op"] == "prompt":
        P.packed_forward(state["shape"], state["Q"], state["K"], state["V"], state["plan"], state["O"], state["lse"])
        return {"O": state["O"], "lse": state["lse"]}
    P.packed_backward(state["shape"], state["Q"], state["K"], state["V"], state["plan"], state["O"], state["lse"],
                      state["dO"], state["delta"], state["dQ"], state["dK"], state["dV"])
    return {"dQ": state["dQ"], "dK": state["dK"], "dV": state["dV"]}


# ---- plain forms -------------------------------------------------------------------------------------------

def _pairs_of(x, rot, layout):
    if layout == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot]
    return x[..., 0:rot:2], x[..., 1:rot:2]


def _plain_rope(st):
    case = st["case"]
    B, N, rot, layout = case["B"], case["N"], case["rot"], case["layout"]
    freq, scale = st["freq"]
    w = torch.tensor(freq, dtype=torch.float64, device="cuda")
    pos = st["pos"]
    if pos is None:
        pos = torch.arange(case["first"], case["first"] + N, device="cuda", dtype=torch.int32).expand(B, N)
    ang = pos.double().unsqueeze(-1) * w  # angles of far positions need the 53 bits
    cos, sin = (torch.cos(ang) * scale).float().unsqueeze(1), (torch.sin(ang) * scale).float().unsqueeze(1)
    if case["inverse"]:
        sin = -sin
    for x, y in ((st["Q"], st["Qo"]), (st["K"], st["Ko"])):
        a, b = _pairs_of(x, rot, layout)
        a, b = a.float(), b.float()
        ya, yb = _pairs_of(y, rot, layout)
        ya.copy_(a * cos - b * sin)
        yb.copy_(a * sin + b * cos)
        y[..., rot:] = x[..., rot:]
    return {"Q": st["Qo"], "K": st["Ko"]}


_ROWS = 2048  # query rows at a time


def _chunks(cu):
    for s, e in zip(cu, cu[1:]):
        for r in range(s, e, _ROWS):
            yield s, r, min(r + _ROWS, e)


def _scores(st, h0, h1, s, r0, r1):
    """Scaled, masked scores [Hkv', G, rows, keys] of the query rows r0..r1 of the sequence that starts at s."""
    Hkv, d = st["K"].shape[0], st["K"].shape[2]
    G = st["Q"].shape[0] // Hkv
    q = st["Q"][h0 * G:h1 * G, r0:r1].float().reshape(h1 - h0, G * (r1 - r0), d)
    k = st["K"][h0:h1, s:r1].float()
    x = torch.bmm(q, k.transpose(1, 2)).reshape(h1 - h0, G, r1 - r0, r1 - s) * (1.0 / math.sqrt(d))
    late = torch.arange(s, r1, device="cuda").unsqueeze(0) > torch.arange(r0, r1, device="cuda").unsqueeze(1)
    return q, k, x.masked_fill_(late, float("-inf"))


def _head_groups(st, rows, keys):
    """kv heads at a time, so that one block of scores stays below 2 GiB."""
    Hkv = st["K"].shape[0]
    G = st["Q"].shape[0] // Hkv
    step = max(1, min(Hkv, (1 << 29) // max(1, G * rows * keys)))
    return [(h, min(h + step, Hkv)) for h in range(0, Hkv, step)]


def _plain_prompt(st):
    Hkv = st["K"].shape[0]
    G = st["Q"].shape[0] // Hkv
    for s, r0, r1 in _chunks(st["cu_host"]):
        for h0, h1 in _head_groups(st, r1 - r0, r1 - s):
            _, _, x = _scores(st, h0, h1, s, r0, r1)
            m = x.amax(dim=-1, keepdim=True)
            p = torch.exp(x - m)
            z = p.sum(dim=-1, keepdim=True)
            o = torch.bmm(p.reshape(h1 - h0, -1, r1 - s), st["V"][h0:h1, s:r1].float())
            o = o.reshape((h1 - h0) * G, r1 - r0, -1) / z.reshape((h1 - h0) * G, r1 - r0, 1)
            st["O"][h0 * G:h1 * G, r0:r1] = o.to(st["O"].dtype)
            st["lse"][h0 * G:h1 * G, r0:r1] = (m + torch.log(z)).reshape((h1 - h0) * G, r1 - r0)
    return {"O": st["O"], "lse": st["lse"]}


def _plain_prompt_grad(st):
    Hkv, T, d = st["K"].shape
    G = st["Q"].shape[0] // Hkv
    dK = torch.zeros((Hkv, T, d), dtype=torch.float32, device="cuda")
    dV = torch.zeros((Hkv, T, d), dtype=torch.float32, device="cuda")
    for s, r0, r1 in _chunks(st["cu_host"]):
        for h0, h1 in _head_groups(st, r1 - r0, r1 - s):
            q, k, x = _scores(st, h0, h1, s, r0, r1)
            n = h1 - h0
            p = torch.softmax(x, dim=-1).reshape(n, -1, r1 - s)
            do = st["dO"][h0 * G:h1 * G, r0:r1].float().reshape(n, -1, d)
            dp = torch.bmm(do, st["V"][h0:h1, s:r1].float().transpose(1, 2))
            ds = p * (dp - (p * dp).sum(dim=-1, keepdim=True)) * (1.0 / math.sqrt(d))
            st["dQ"][h0 * G:h1 * G, r0:r1] = torch.bmm(ds, k).reshape(n * G, r1 - r0, d).to(st["dQ"].dtype)
            dK[h0:h1, s:r1] += torch.bmm(ds.transpose(1, 2), q)
            dV[h0:h1, s:r1] += torch.bmm(p.transpose(1, 2), do)
    e = st["cu_host"][-1]
    st["dK"][:, :e] = dK[:, :e].to(st["dK"].dtype)
    st["dV"][:, :e] = dV[:, :e].to(st["dV"].dtype)
    return {"dQ": st["dQ"], "dK": st["dK"], "dV": st["dV"]}


def _plain_tree(st):
    B, Hq, T, d = st["Q"].shape
    Hkv = st["K"].shape[1]
    G = Hq // Hkv
    # sees[b][t][u]: drafted token u is t or one of its ancestors
    sees = torch.eye(T, dtype=torch.bool, device="cuda").expand(B, T, T).clone()
    up = st["parent"].long()
    for t in range(T):
        own_row = sees[:, t].clone()
        p = up[:, t]
        above = torch.gather(sees, 1, p.clamp(min=0).reshape(B, 1, 1).expand(B, 1, T))[:, 0]
        sees[:, t] = own_row | (above & (p >= 0).unsqueeze(1))
    for b, n in enumerate(st["lens_host"]):
        q = st["Q"][b].float().reshape(Hkv, G * T, d)
        x = torch.bmm(q, st["K"][b, :, :n + T].float().transpose(1, 2)) * (1.0 / math.sqrt(d))
        x = x.reshape(Hkv, G, T, n + T)
        x[..., n:].masked_fill_(~sees[b], float("-inf"))
        m = x.amax(dim=-1, keepdim=True)
        p = torch.exp(x - m)
        z = p.sum(dim=-1, keepdim=True)
        o = torch.bmm(p.reshape(Hkv, G * T, n + T), st["V"][b, :, :n + T].float()).reshape(Hkv, G, T, d) / z
        st["O"][b] = o.reshape(Hq, T, d).to(st["O"].dtype)
        st["lse"][b] = (m + torch.log(z)).reshape(Hq, T)
    return {"O": st["O"], "lse": st["lse"]}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------

def _softmax64(scores, visible):
    """(probabilities, log-sum-exp) of scores where visible."""
    scores = torch.where(visible, scores, torch.full_like(scores, -math.inf))
    lse = torch.logsumexp(scores, dim=-1)
    return torch.exp(scores - lse.unsqueeze(-1)), lse


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(dict(case, op="prompt") if case["op"] == "prompt_grad" else case, seed)
        if case["op"] == "prompt_grad":
            # the gradient's extra input comes after Q, K and V in the generator's stream
            st = {k: st[k] for k in ("Q", "K", "V", "cu_host")}
            gen = _generator(seed)
            dt, T = _DT[case["dtype"]], st["Q"].shape[1]
            for H, off in ((case["Hq"], False), (case["Hkv"], True), (case["Hkv"], False)):
                _normal(gen, case["order"], 1, H, T, case["d"], dt, offsets=off)
            st["dO"] = _normal(gen, case["order"], 1, case["Hq"], T, case["d"], dt)[0]
    finally:
        own = keep
    return {"rope": _exact_rope, "prompt": _exact_prompt, "prompt_grad": _exact_prompt_grad,
            "tree": _exact_tree}[case["op"]](case, st)


def _exact_rope(case, st):
    # every pair as a complex number, turned by exp(i pos w)
    w, c = _frequencies(case)
    w = torch.tensor(w, dtype=torch.float64, device="cuda")
    pos = st["pos"]
    if pos is None:
        pos = case["first"] + torch.arange(case["N"], device="cuda").expand(case["B"], -1)
    turn = pos.double()[:, None, :, None] * w * (-1.0 if case["inverse"] else 1.0)
    out = {}
    for name in ("Q", "K"):
        x = st[name].double()
        n = case["rot"] // 2
        if case["layout"] == "half":
            i, j = torch.arange(n, device="cuda"), torch.arange(n, device="cuda") + n
        else:
            i, j = 2 * torch.arange(n, device="cuda"), 2 * torch.arange(n, device="cuda") + 1
        z = torch.complex(x[..., i], x[..., j]) * torch.polar(torch.full_like(turn, c), turn)
        x[..., i], x[..., j] = z.real, z.imag
        out[name] = x
    return out


def _exact_prompt(case, st):
    Q, K, V, cu = st["Q"], st["K"], st["V"], st["cu_host"]
    O = torch.zeros(Q.shape, dtype=torch.float64, device="cuda")
    L = torch.zeros(Q.shape[:2], dtype=torch.float64, device="cuda")
    for s, e in zip(cu, cu[1:]):
        t = torch.arange(e - s, device="cuda")
        visible = t[:, None] >= t[None, :]
        for h in range(Q.shape[0]):
            g = h * K.shape[0] // Q.shape[0]
            p, lse = _softmax64(Q[h, s:e].double() @ K[g, s:e].double().T / math.sqrt(case["d"]), visible)
            O[h, s:e], L[h, s:e] = p @ V[g, s:e].double(), lse
    return {"O": O, "lse": L}


def _exact_prompt_grad(case, st):
    Q, K, V, dO, cu = st["Q"], st["K"], st["V"], st["dO"], st["cu_host"]
    scale = 1.0 / math.sqrt(case["d"])
    dQ, dK, dV = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (Q, K, V))
    for s, e in zip(cu, cu[1:]):
        t = torch.arange(e - s, device="cuda")
        visible = t[:, None] >= t[None, :]
        for h in range(Q.shape[0]):
            g = h * K.shape[0] // Q.shape[0]
            q, k, v, do = Q[h, s:e].double(), K[g, s:e].double(), V[g, s:e].double(), dO[h, s:e].double()
            p, _ = _softmax64(q @ k.T * scale, visible)
            o = p @ v
            dV[g, s:e] += p.T @ do
            p *= do @ v.T - (do * o).sum(dim=1, keepdim=True)
            dQ[h, s:e] = p @ k * scale
            dK[g, s:e] += p.T @ q * scale
    return {"dQ": dQ, "dK": dK, "dV": dV}


def _exact_tree(case, st):
    Q, K, V = st["Q"], st["K"], st["V"]
    B, Hq, T, d = Q.shape
    O = torch.empty(Q.shape, dtype=torch.float64, device="cuda")
    L = torch.empty(Q.shape[:3], dtype=torch.float64, device="cuda")
    parents = st["parent"].tolist()
    for b, n in enumerate(st["lens_host"]):
        visible = torch.zeros((T, n + T), dtype=torch.bool)
        visible[:, :n] = True
        for t in range(T):
            u = t
            while u >= 0:
                visible[t, n + u] = True
                u = parents[b][u]
        visible = visible.cuda()
        for h in range(Hq):
            g = h * K.shape[1] // Hq
            p, L[b, h] = _softmax64(Q[b, h].double() @ K[b, g, :n + T].double().T / math.sqrt(d), visible)
            O[b, h] = p @ V[b, g, :n + T].double()
    return {"O": O, "lse": L}
