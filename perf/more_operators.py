"""The attention layer of a token decoder and the step that trains it, as cases to be measured:
attention (whole grids, and single tokens over a cache), its gradient, rotary positions with
several axes, and an AdamW step over many tensors with its states in 32 or in 8 bits.

A case is a dict of plain values; `op` names the operator.  `run` computes it either in
elementary torch operations (`own` false) or through the package's entry points (`own`
true); `exact` computes it from the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
SIZE = {"float32": 4, "float16": 2, "bfloat16": 2}
INF = float("inf")
BLOCK = 256  # elements that share a scale where a state is held in 8 bits
TOP = 448.0  # the largest e4m3 value
LEAST = 2.0 ** -126  # the smallest scale
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.01, step=10, grad_scale=1.0 / 1024)


# ------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------
def attend(op, dtype, n, tq, tk, heads, kv_heads, width, causal=False, lengths=False):
    return {"op": op, "dtype": dtype, "n": n, "tq": tq, "tk": tk, "heads": heads, "kv_heads": kv_heads, "width": width,
            "causal": causal, "lengths": lengths}


def rotary(dtype, n, dims, heads, width, sections, far=False, whole=False, interleaved=False, inverse=False):
    return {"op": "rotary", "dtype": dtype, "n": n, "dims": dims, "heads": heads, "width": width, "sections": sections,
            "far": far, "whole": whole, "interleaved": interleaved, "inverse": inverse}


def adamw(dtype, grad, bits, pairs, rows, width, copy=""):
    return {"op": "adamw", "dtype": dtype, "grad": grad, "bits": bits, "pairs": pairs, "rows": rows, "width": width,
            "copy": copy}


def listed():
    return [
        # the next code of 8 sequences over caches of up to 4096 positions: latency counts
        dict(attend("attend", "float16", 8, 1, 4096, 8, 2, 64, causal=True, lengths=True), name="attend_one_token"),
        # all positions of the 2-D decoder layer's input: 8 images of 64 x 64, 512 channels in 8 heads
        dict(attend("attend", "float16", 8, 4096, 4096, 8, 8, 64), name="attend_decoder"),
        # the codes of long sequences seen causally, shared key heads, an odd length
        dict(attend("attend", "bfloat16", 2, 8191, 8191, 16, 4, 128, causal=True), name="attend_causal_shared"),
        # texts of different lengths that an odd number of queries look at, float32, one text empty
        dict(attend("attend", "float32", 3, 77, 1001, 5, 5, 40, lengths=True), name="attend_odd"),
        # the gradient over the 2-D decoder layer's input
        dict(attend("attend_grad", "float16", 8, 4096, 4096, 8, 8, 64), name="attend_grad_decoder"),
        # the gradient of causal training with shared key heads, an odd length
        dict(attend("attend_grad", "bfloat16", 1, 4097, 4097, 16, 4, 128, causal=True), name="attend_grad_causal_shared"),
        # a small float32 layer over a padded batch
        dict(attend("attend_grad", "float32", 4, 257, 257, 3, 3, 36, lengths=True), name="attend_grad_odd"),
        # queries and keys of the next code of 8 sequences, far into them: latency counts
        dict(rotary("float16", 8, "1", 10, 64, "8x12x12", far=True), name="rotary_one_token"),
        # the 3-D layer's input, 2 clips of 16 x 32 x 32, by time, height and width
        dict(rotary("bfloat16", 2, "16x32x32", 20, 128, "16x24x24", inverse=True), name="rotary_clip"),
        # the token decoder example's parameters and a 16-bit copy of them
        dict(adamw("float32", "float16", 32, 3, 512, 64, copy="float16"), name="adamw_small"),
        # 48 tensors, 50 million parameters, 32-bit states
        dict(adamw("float32", "bfloat16", 32, 24, 4096, 512, copy="bfloat16"), name="adamw_32_bits"),
        # the same parameters in 16 bits with 8-bit states
        dict(adamw("bfloat16", "bfloat16", 8, 24, 4096, 511), name="adamw_8_bits"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


MOST_PAIRS = 8 * 8 * 4096 * 4096


def draw(rng):
    op = rng.choice(["attend", "attend", "attend_cache", "attend_cache", "attend_grad", "attend_grad", "rotary", "rotary",
                     "adamw", "adamw"])
    dtype = rng.choice(["float16", "bfloat16", "float16", "bfloat16", "float32"])
    width = rng.choice([64, 64, 128, 128, 32, 96, 256, rng.randint(4, 32) * 4, rng.randint(9, 160)])
    if op.startswith("attend"):
        kv_heads = rng.choice([1, 2, 4, 8, 3])
        heads = kv_heads * rng.choice([1, 1, 2, 4, 5])
        n = _log(rng, 1, 16)
        if op == "attend_cache":  # a few new tokens over what went before
            tq = rng.choice([1, 1, 1, 2, 5, 16])
            tk = _log(rng, 16, min(65536, (1 << 28) // (n * kv_heads * width)))
            return attend("attend", dtype, n, tq, tk, heads, kv_heads, width, causal=True, lengths=True)
        side = math.sqrt(MOST_PAIRS * min(1.0, 64 / width) * (0.05 if dtype == "float32" else 1.0) / (n * heads))
        tk = _log(rng, 1, min(8192, side))
        tq = tk if rng.random() < 0.7 else _log(rng, 1, min(8192, side))
        causal = tq <= tk and rng.random() < 0.5
        # a single visible key's gradient of the query is nothing but cancellation
        if op == "attend_grad":
            tk = max(tk, 16)
            tq = tk if causal else tq
        return attend(op, dtype, n, tq, tk, heads, kv_heads, width, causal=causal, lengths=not causal and rng.random() < 0.4)
    if op == "rotary":
        axes = rng.choice([1, 2, 3, 3])
        heads = rng.choice([1, 3, 8, 10, 16, 20])
        width = max(width, 2 * axes)
        pairs = width // 2 - (width // 8 if rng.random() < 0.3 else 0)
        pairs = max(pairs, axes)
        cut = [pairs // axes] * axes
        cut[0] += pairs - sum(cut)
        n = _log(rng, 1, 16)
        positions = _log(rng, 1, min(65536, (1 << 26) // (n * heads * width)))
        side = max(1, int(round(positions ** (1.0 / axes))))
        dims = [side] * (axes - 1) + [max(1, positions // side ** (axes - 1))]
        return rotary(dtype, n, "x".join(map(str, dims)), heads, width, "x".join(map(str, cut)), far=rng.random() < 0.3,
                      whole=rng.random() < 0.5, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)
    bits = rng.choice([32, 8])
    rows, wide = _log(rng, 1, 4096), _log(rng, 1, 2048)
    pairs = _log(rng, 1, max(1, min(24, 48_000_000 // ((rows + 1) * wide))))
    return adamw(dtype, rng.choice(["float32", dtype]), bits, pairs, rows, wide,
                 copy=rng.choice(["", "float16", "bfloat16"]) if dtype == "float32" else "")


def _numbers(text):
    return [int(s) for s in text.split("x")]


def _tensors(case):
    """(elements, first place in the flat buffers, weight decay) of each tensor: a matrix and a vector a pair."""
    sizes = [s for _ in range(case["pairs"]) for s in (case["rows"] * case["width"], case["width"])]
    at, found = 0, []
    for k, size in enumerate(sizes):
        found.append((size, at, 0.0 if k % 2 else HYPER["decay"]))
        at += -(-size // BLOCK) * BLOCK
    return found, at


# ------------------------------------------------------------------------------------
# the inputs
# ------------------------------------------------------------------------------------
def _attend_state(case, gen, dev):
    dtype, n, tq, tk = TYPES[case["dtype"]], case["n"], case["tq"], case["tk"]
    h, hk, d = case["heads"], case["kv_heads"], case["width"]
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    if tq == tk:  # one projection left queries, keys and values side by side
        packed = randn(n, tk, h + 2 * hk, d)
        packed[:, :, :h] *= 0.5 + 1.5 * torch.rand((h, 1), generator=gen, device=dev)
        packed = packed.to(dtype)
        state = {"q": packed[:, :, :h], "k": packed[:, :, h:h + hk], "v": packed[:, :, h + hk:]}
    else:
        gain = 0.5 + 1.5 * torch.rand((h, 1), generator=gen, device=dev)
        state = {"q": (randn(n, tq, h, d) * gain).to(dtype), "k": randn(n, tk, hk, d).to(dtype),
                 "v": randn(n, tk, hk, d).to(dtype)}
    state.update(case=case, lengths=None, starts=None)
    if case["lengths"]:
        least = min(tq, tk) if case["causal"] else 0
        lengths = torch.randint(least, tk + 1, (n,), generator=gen, device=dev, dtype=torch.int32)
        lengths[0] = tk
        if n > 2 and not case["causal"]:
            lengths[-1] = 0  # nothing to look at
        state["lengths"] = lengths
        if case["causal"]:
            state["starts"] = lengths - tq
    if case["op"] == "attend_grad":
        state["dout"] = randn(n, tq, h, d).to(dtype)
        state["out"], state["lse"] = _plain_attend(state)  # the forward pass left them
    return state


def _rotary_state(case, gen, dev):
    dims, axes = _numbers(case["dims"]), len(_numbers(case["sections"]))
    dims = dims if len(dims) == axes else [1] * (axes - len(dims)) + dims
    grid = torch.stack(torch.meshgrid(*(torch.arange(s, device=dev) for s in dims), indexing="ij"), -1).reshape(1, -1, axes)
    if case["far"]:  # every sequence at a place of its own
        grid = grid + torch.randint(0, 1 << 20, (case["n"], 1, axes), generator=gen, device=dev)
    positions = grid.to(torch.int32).expand(case["n"], -1, -1)
    # what turns (queries and keys) lies in front of what does not (values)
    heads = case["heads"] + max(1, case["heads"] // 4)
    x = torch.randn((case["n"], grid.shape[1], heads, case["width"]), generator=gen, device=dev).to(TYPES[case["dtype"]])
    return {"x": x[:, :, :case["heads"]], "positions": positions}


def _adamw_state(case, gen, dev):
    tensors, size = _tensors(case)
    dtype, grad = TYPES[case["dtype"]], TYPES[case["grad"]]
    used = torch.zeros(size, dtype=torch.bool, device=dev)
    for count, at, _ in tensors:
        used[at:at + count] = True
    randn = lambda: torch.where(used, torch.randn(size, generator=gen, device=dev), 0.0)  # noqa: E731
    # gradients of a loss that was scaled up; every block of weights has a spread of its own
    spread = torch.exp(1.5 * torch.randn(size // BLOCK, generator=gen, device=dev)).repeat_interleave(BLOCK) * 1e-3
    state = {"p": randn().mul_(0.05).to(dtype), "g": (randn() * spread / HYPER["grad_scale"]).to(grad)}
    m, v = randn() * spread * 0.3, (randn() * spread).square() * 0.9 + (spread * used).square() * 0.1
    if case["bits"] == 32:
        state["m"], state["v"] = m, v
    else:
        state["m"], state["m_scale"] = _plain_code(m.reshape(-1, BLOCK))
        state["v"], state["v_scale"] = _plain_code(v.reshape(-1, BLOCK).sqrt(), True)
    if case["copy"]:
        state["copy"] = torch.zeros(size, dtype=TYPES[case["copy"]], device=dev)
    decay = torch.tensor([d for count, _, d in tensors for _ in range(-(-count // BLOCK))], dtype=torch.float32)
    state["decay"] = decay.to(dev)[:, None]
    state["step"] = torch.tensor([HYPER["step"]], dtype=torch.int64, device=dev)
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    make = {"rotary": _rotary_state, "adamw": _adamw_state}.get(case["op"], _attend_state)
    state = {"case": case, **make(case, gen, dev)}
    if own:
        state["call"] = _own_call(state)
    return state


# ------------------------------------------------------------------------------------
# through the package
# ------------------------------------------------------------------------------------
def _own_call(state):
    """The call that a program with these buffers keeps and repeats."""
    import transposed_convolution_amd as T

    case = state["case"]
    if case["op"] in ("attend", "attend_grad"):
        mask = dict(causal=case["causal"], lengths=state["lengths"], starts=state["starts"])
        if case["op"] == "attend":
            return T.PreparedCall(T.attention_nd, state["q"], state["k"], state["v"], **mask)
        return T.PreparedCall(T.attention_backward_nd, state["dout"], state["q"], state["k"], state["v"], state["out"],
                              state["lse"], **mask)
    if case["op"] == "rotary":
        return T.PreparedCall(T.rotary_nd, state["x"], state["positions"], _numbers(case["sections"]),
                              whole_ladder=case["whole"], interleaved=case["interleaved"], inverse=case["inverse"])
    tensors, _ = _tensors(case)
    cut = lambda t: [t.reshape(-1)[at:at + n] for n, at, _ in tensors]  # noqa: E731
    scales = lambda t: [t[at // BLOCK:-(-(at + n) // BLOCK)] for n, at, _ in tensors]  # noqa: E731
    options = dict(lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"], step=state["step"],
                   weight_decay=[d for _, _, d in tensors], grad_scale=HYPER["grad_scale"])
    if case["bits"] == 8:
        options.update(m_scales=scales(state["m_scale"]), v_scales=scales(state["v_scale"]))
    if case["copy"]:
        options.update(copies=cut(state["copy"]))
    return T.PreparedCall(T.adamw_nd, cut(state["p"]), cut(state["g"]), cut(state["m"]), cut(state["v"]), **options)


def run(state):
    op = state["case"]["op"]
    if own:
        made = state["call"]()
        return _updated(state) if op == "adamw" else made
    return {"attend": _plain_attend, "attend_grad": _plain_attend_grad, "rotary": _plain_rotary, "adamw": _plain_adamw}[op](state)


def _updated(state):
    return {k: state[k] for k in ("p", "m", "v", "m_scale", "v_scale", "copy") if k in state}


# ------------------------------------------------------------------------------------
# the plain forms: elementary torch operations in 32 bits, rounded once at the end
# ------------------------------------------------------------------------------------
def _by_kv_head(t, kv_heads):
    """(N, T, H, D) as (N, Hkv, G T, D) in 32 bits: the query heads of a key head one after the other."""
    n, tokens, heads, d = t.shape
    return t.float().permute(0, 2, 1, 3).reshape(n, kv_heads, heads // kv_heads * tokens, d)


def _by_token(t, heads, dtype):
    n, d = t.shape[0], t.shape[3]
    return t.reshape(n, heads, -1, d).permute(0, 2, 1, 3).to(dtype).contiguous()


def _plain_hidden(state, rows):
    """Which keys a query does not see, (N or 1, 1, G Tq, Tk), or None."""
    case, dev = state["case"], state["q"].device
    j = torch.arange(case["tk"], device=dev)
    hidden = None
    if case["causal"]:
        i = torch.arange(case["tq"], device=dev)
        start = state["starts"][:, None] if state["starts"] is not None else case["tk"] - case["tq"]
        last = (i + start).reshape(-1, case["tq"]).repeat(1, rows // case["tq"])
        hidden = j > last[:, None, :, None]
    if state["lengths"] is not None:
        behind = j >= state["lengths"][:, None, None, None]
        hidden = behind if hidden is None else hidden | behind
    return hidden


def _plain_scores(state):
    hk = state["case"]["kv_heads"]
    q, k = _by_kv_head(state["q"], hk), _by_kv_head(state["k"], hk)
    s = (q @ k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(state["case"]["width"]))
    hidden = _plain_hidden(state, q.shape[2])
    return q, k, s if hidden is None else s.masked_fill_(hidden, -INF)


def _plain_attend(state):
    case = state["case"]
    _, _, s = _plain_scores(state)
    top = s.amax(3, keepdim=True)
    top = torch.where(top == -INF, 0.0, top)  # a row that sees nothing
    p = s.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    out = (p @ _by_kv_head(state["v"], case["kv_heads"])) / torch.where(total == 0.0, 1.0, total)
    lse = (top + total.log()).reshape(case["n"], case["heads"], case["tq"])
    return _by_token(out, case["heads"], state["q"].dtype), lse


def _plain_attend_grad(state):
    case, hk = state["case"], state["case"]["kv_heads"]
    q, k, s = _plain_scores(state)
    lse = state["lse"].reshape(case["n"], hk, -1, 1)
    p = s.sub_(torch.where(lse == -INF, 0.0, lse)).exp_()
    do, v = _by_kv_head(state["dout"], hk), _by_kv_head(state["v"], hk)
    dv = p.transpose(2, 3).contiguous() @ do
    delta = (do * _by_kv_head(state["out"], hk)).sum(3, keepdim=True)
    ds = (do @ v.transpose(2, 3).contiguous()).sub_(delta).mul_(p).mul_(1.0 / math.sqrt(case["width"]))
    dq, dk = ds @ k, ds.transpose(2, 3).contiguous() @ q
    dtype = state["q"].dtype
    return _by_token(dq, case["heads"], dtype), _by_token(dk, hk, dtype), _by_token(dv, hk, dtype)


def _frequencies(case, dev):
    """Angle a position of every pair (float64), and the axis it goes by."""
    sections = _numbers(case["sections"])
    total = sum(sections)
    of = torch.arange(total, device=dev, dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=dev), torch.tensor(sections, device=dev))
    if case["whole"]:
        part = of / total
    else:
        size = torch.tensor(sections, device=dev, dtype=torch.float64)
        part = (of - (size.cumsum(0) - size)[axis]) / size[axis]
    return torch.exp(-math.log(10000.0) * part), axis


def _plain_rotary(state):
    case, x = state["case"], state["x"]
    inv, axis = _frequencies(case, x.device)
    angle = (state["positions"].double()[:, :, axis] * inv)[:, :, None]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    s = -s if case["inverse"] else s
    total = inv.numel()
    v = x.float()
    if case["interleaved"]:
        a, b = v[..., 0:2 * total:2], v[..., 1:2 * total:2]
        y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(3)
    else:
        a, b = v[..., :total], v[..., total:2 * total]
        y = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((y, v[..., 2 * total:]), -1).to(x.dtype)


def _plain_code(t, root=False):
    """Blocks (rows) of `t` as e4m3 values and a scale each.  A positive root never becomes 0: what is
    divided by it would grow without bound."""
    scale = (t.abs().amax(1, keepdim=True) / TOP).clamp(min=LEAST)
    code = t / scale
    if root:
        code = torch.where(t > 0.0, code.clamp(min=2.0 ** -9), code)
    return code.to(torch.float8_e4m3fn).reshape(-1), scale.reshape(-1)


def _plain_adamw(state):
    case, h = state["case"], HYPER
    step = state["step"].double()
    first, second = (1.0 - h["beta1"] ** step), (1.0 - h["beta2"] ** step)
    rate, root = (h["lr"] / first).float(), (1.0 / second.sqrt()).float()
    rows = lambda k: state[k].float().reshape(-1, BLOCK)  # noqa: E731
    g = rows("g") * h["grad_scale"]
    m, v = rows("m"), rows("v")
    if case["bits"] == 8:
        m, v = m * state["m_scale"][:, None], (v * state["v_scale"][:, None]).square()
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + g.square() * (1.0 - h["beta2"])
    p = rows("p") * (1.0 - h["lr"] * state["decay"]) - m / (v.sqrt() * root + h["eps"]) * rate
    state["p"].copy_(p.reshape(-1))
    if "copy" in state:
        state["copy"].copy_(p.reshape(-1))
    if case["bits"] == 32:
        state["m"].copy_(m.reshape(-1))
        state["v"].copy_(v.reshape(-1))
    else:
        state["m"], state["m_scale"] = _plain_code(m)
        state["v"], state["v_scale"] = _plain_code(v.sqrt(), True)
    return _updated(state)


# ------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------
def _exact_head(state, n, h):
    """Probabilities (Tq, Tk), log sums, and q, k, v of one image's head."""
    case = state["case"]
    shared = h // (case["heads"] // case["kv_heads"])
    q, k, v = state["q"][n, :, h].double(), state["k"][n, :, shared].double(), state["v"][n, :, shared].double()
    s = torch.matmul(q, k.t().contiguous()) / math.sqrt(case["width"])
    length = case["tk"] if state["lengths"] is None else int(state["lengths"][n])
    seen = torch.zeros_like(s, dtype=torch.bool)
    seen[:, :length] = True
    if case["causal"]:
        start = case["tk"] - case["tq"] if state["starts"] is None else int(state["starts"][n])
        seen &= torch.ones_like(seen).tril(start)
    s = torch.where(seen, s, -INF)
    lse = torch.logsumexp(s, 1)
    p = torch.where(seen, torch.exp(s - torch.where(lse == -INF, 0.0, lse)[:, None]), 0.0)
    return p, lse, q, k, v


def _exact_attend(state):
    case = state["case"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device=state["q"].device)
    lse = torch.zeros((case["n"], case["heads"], case["tq"]), dtype=torch.float64, device=out.device)
    for n in range(case["n"]):
        for h in range(case["heads"]):
            p, lse[n, h], _, _, v = _exact_head(state, n, h)
            out[n, :, h] = torch.matmul(p, v)
    return out, lse


def _exact_attend_grad(state):
    case = state["case"]
    dq, dk, dv = (torch.zeros(state[k].shape, dtype=torch.float64, device=state["q"].device) for k in "qkv")
    for n in range(case["n"]):
        for h in range(case["heads"]):
            p, _, q, k, v = _exact_head(state, n, h)
            do = state["dout"][n, :, h].double()
            dp = torch.matmul(do, v.t().contiguous())
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(case["width"])
            shared = h // (case["heads"] // case["kv_heads"])
            dq[n, :, h] = torch.matmul(ds, k)
            dk[n, :, shared] += torch.matmul(ds.t().contiguous(), q)
            dv[n, :, shared] += torch.matmul(p.t().contiguous(), do)
    return dq, dk, dv


def _exact_rotary(state):
    case, x = state["case"], state["x"].double()
    sections = _numbers(case["sections"])
    total, y, pair = sum(sections), x.clone(), 0
    for axis, size in enumerate(sections):
        for j in range(size):
            inv = 10000.0 ** (-(pair / total if case["whole"] else j / size))
            z = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device),
                            state["positions"][:, :, axis, None].double() * (-inv if case["inverse"] else inv))
            a, b = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + total)
            y[..., a] = x[..., a] * z.real - x[..., b] * z.imag
            y[..., b] = x[..., a] * z.imag + x[..., b] * z.real
            pair += 1
    return y


def _exact_code(t, root=False):
    """e4m3 values (4 significant bits, steps of at least 2^-9) and the scale of every row, in 64 bits."""
    scale = torch.clamp(t.abs().max(1, keepdim=True).values / TOP, min=LEAST)
    x = t / scale
    step = torch.exp2(torch.clamp(torch.frexp(x).exponent - 1, min=-6).double() - 3)
    code = torch.round(x / step) * step
    if root:
        code = torch.where((t > 0) & (code == 0), 2.0 ** -9, code)
    return code.flatten(), scale.flatten()


def _exact_adamw(state):
    case, h = state["case"], HYPER
    blocks = lambda t: t.double().reshape(-1, BLOCK)  # noqa: E731
    m, v, g = blocks(state["m"]), blocks(state["v"]), blocks(state["g"]) * h["grad_scale"]
    if case["bits"] == 8:
        m, v = m * blocks(state["m_scale"].repeat_interleave(BLOCK)), (v * blocks(state["v_scale"].repeat_interleave(BLOCK))) ** 2
    m, v = torch.lerp(g, m, h["beta1"]), torch.lerp(g * g, v, h["beta2"])
    mh, vh = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p = blocks(state["p"])
    p = (p - h["lr"] * (mh / (vh ** 0.5 + h["eps"]) + state["decay"].double() * p)).flatten()
    made = {"p": p, "m": m.flatten(), "v": v.flatten()}
    if case["bits"] == 8:
        made["m"], made["m_scale"] = _exact_code(m)
        made["v"], made["v_scale"] = _exact_code(v ** 0.5, True)
    if case["copy"]:
        made["copy"] = p
    return made


def exact(case, seed):
    state = prepare(case, seed)
    return {"attend": _exact_attend, "attend_grad": _exact_attend_grad, "rotary": _exact_rotary,
            "adamw": _exact_adamw}[case["op"]](state)


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def _pairs(case):
    """Query-key pairs that are seen, about: lengths are drawn evenly up to the whole."""
    tq, tk = case["tq"], case["tk"]
    seen = tk * (0.5 if case["lengths"] else 1.0)
    if case["causal"]:
        seen = (seen if case["lengths"] else tk) - (tq - 1) / 2
    return case["n"] * case["heads"] * tq * max(1.0, seen)


def work(case):
    if case["op"] == "adamw":
        count = sum(n for n, _, _ in _tensors(case)[0])
        each = 2 * SIZE[case["dtype"]] + SIZE[case["grad"]] + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": count * (each + (SIZE[case["copy"]] if case["copy"] else 0)), "flops": 15 * count}
    size = SIZE[case["dtype"]]
    if case["op"] == "rotary":
        tokens = case["n"] * math.prod(_numbers(case["dims"]))
        axes = len(_numbers(case["sections"]))
        count = tokens * case["heads"] * case["width"]
        return {"bytes": 2 * count * size + tokens // (1 if case["far"] else case["n"]) * axes * 4, "flops": 3 * count}
    rows = case["n"] * case["heads"] * case["tq"]
    kept = 0.5 if case["lengths"] else 1.0
    keys = case["n"] * case["kv_heads"] * case["tk"] * case["width"] * size * 2
    if case["op"] == "attend":
        return {"bytes": keys * kept + 2 * rows * case["width"] * size + 4 * rows, "flops": 4 * _pairs(case) * case["width"]}
    return {"bytes": keys * (1 + kept) + 4 * rows * case["width"] * size + 4 * rows, "flops": 10 * _pairs(case) * case["width"]}
