"""The operators around the transposed convolution in a decoder, as cases to be measured:
channels-last group norm with an activation (forward and gradient), dropout from a
counter-based generator, and the embedding lookup (forward and gradient).

A case is a dict of plain values; `op` names the operator.  `run` computes it either in
elementary torch operations (`own` false) or through the package's entry points (`own`
true); `exact` computes it from the definition in 64 bits.
"""
import functools
import math

import numpy as np
import torch

own = False

TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
SIZE = {"float32": 4, "float16": 2, "bfloat16": 2}
MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------
def group_norm(op, dtype, n, c, dims, groups, act="silu", p=0.0, params="float32"):
    return {"op": op, "dtype": dtype, "n": n, "c": c, "dims": dims, "groups": groups, "act": act, "p": p,
            "params": params}


def dropout(dtype, count, p, residual):
    return {"op": "dropout", "dtype": dtype, "count": count, "p": p, "residual": residual}


def embedding(op, dtype, tokens, rows, width, ids="int64", padding=False):
    return {"op": op, "dtype": dtype, "tokens": tokens, "rows": rows, "width": width, "ids": ids, "padding": padding}


def listed():
    return [
        # one 8 x 8 latent before the first upsampling layer, a single image: latency counts
        dict(group_norm("norm", "float16", 1, 256, "8x8", 32), name="norm_one_latent"),
        # the output of the 2-D decoder layer (512 -> 256 channels, 64 x 64 -> 128 x 128, 8 images)
        dict(group_norm("norm", "float16", 8, 256, "128x128", 32), name="norm_decoder"),
        # a 1-D decoder in float32: 36 channels in groups of 9, an odd length, dropout inside
        dict(group_norm("norm", "float32", 4, 36, "1001", 4, p=0.1), name="norm_1d_odd"),
        # the gradient at the decoder layer's output, with the dropout of training
        dict(group_norm("norm_grad", "float16", 8, 256, "128x128", 32, p=0.1), name="norm_grad_decoder"),
        # the gradient at the 3-D stride-2 layer's output (64 channels, 32 x 64 x 64), bfloat16 training
        dict(group_norm("norm_grad", "bfloat16", 2, 64, "32x64x64", 16, params="bfloat16"), name="norm_grad_3d"),
        # dropout of one small latent: latency counts
        dict(dropout("float16", 256 * 8 * 8, 0.1, False), name="dropout_one_latent"),
        # a residual branch at the decoder layer's output
        dict(dropout("float16", 8 * 256 * 128 * 128, 0.1, True), name="dropout_residual_decoder"),
        # an odd number of float32 values, half of them dropped
        dict(dropout("float32", 4 * 32 * 770 * 9 + 5, 0.5, False), name="dropout_odd"),
        # the next token of a serving loop, one row of a codebook
        dict(embedding("embed", "float16", 1, 8192, 512), name="embed_one_token"),
        # the code images of the 2-D decoder layer's input (8 x 64 x 64 tokens, 512 channels)
        dict(embedding("embed", "float16", 8 * 64 * 64, 16384, 512), name="embed_decoder"),
        # their gradient: code use is skewed, the most used rows take thousands of tokens
        dict(embedding("embed_grad", "float16", 8 * 64 * 64, 16384, 512), name="embed_grad_decoder"),
        # a class or text table of odd width: few tokens, many of them padding
        dict(embedding("embed_grad", "float32", 257, 1025, 77, ids="int32", padding=True), name="embed_grad_odd"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _dims(rng, rank, positions):
    """`rank` axes of about `positions` positions in all, any sizes."""
    sizes, left = [], max(1, positions)
    for axis in range(rank - 1):
        near = left ** (1.0 / (rank - axis))
        sizes.append(max(1, min(left, int(round(near * math.exp(rng.uniform(-0.4, 0.4)))))))
        left = max(1, left // sizes[-1])
    return "x".join(str(s) for s in sizes + [left])


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "dropout", "embed", "embed_grad"])
    dtype = rng.choice(["float16", "float16", "bfloat16", "float32"])
    most = (1 << 25) * 2 // SIZE[dtype]
    if op in ("norm", "norm_grad"):
        n = _log(rng, 1, 16)
        groups = rng.choice([1, 2, 4, 8, 16, 32, 32])
        c = groups * (rng.choice([1, 2, 4, 8, 16, 32]) if rng.random() < 0.6 else rng.randint(1, 24))
        # at least 16 values a group: the gradient through the statistics of fewer is nearly all cancellation
        fewest = -(-16 * groups // c)
        positions = _log(rng, fewest, max(fewest, most // (n * c)))
        act = rng.choice(["silu", "silu", "identity"] if op == "norm_grad" else ["silu", "silu", "identity", "relu"])
        return group_norm(op, dtype, n, c, _dims(rng, rng.randint(1, 3), positions), groups, act=act,
                          p=rng.choice([0.0, 0.0, 0.1, 0.3]), params=rng.choice(["float32", dtype]))
    if op == "dropout":
        return dropout(dtype, _log(rng, 1, most), rng.choice([0.05, 0.1, 0.2, 0.5]), rng.random() < 0.5)
    width = _log(rng, 1, 1024)
    tokens = _log(rng, 1, min(65536, (1 << 24) // width))
    rows = _log(rng, 2, min(65536, (1 << 24) // width))
    return embedding(op, dtype, tokens, rows, width, ids=rng.choice(["int64", "int32"]),
                     padding=op == "embed_grad" and rng.random() < 0.3)


def _shape(case):
    return (case["n"], case["c"]) + tuple(int(s) for s in case["dims"].split("x"))


# ------------------------------------------------------------------------------------
# the inputs
# ------------------------------------------------------------------------------------
def _channels_last(t):
    """(N, D.., C) storage as the logical (N, C, D..)."""
    return t.movedim(-1, 1)


def _norm_state(case, seed, gen, dev):
    dtype, shape = TYPES[case["dtype"]], _shape(case)
    n, c, dims = shape[0], shape[1], shape[2:]
    stored = (n,) + dims + (c,)
    # a convolution's outputs: every channel has a mean (its bias) and a spread of its own
    x = torch.randn(stored, generator=gen, device=dev)
    x = x * (0.5 + torch.rand(c, generator=gen, device=dev)) + torch.randn(c, generator=gen, device=dev)
    params = TYPES[case["params"]]
    state = {"x": _channels_last(x.to(dtype)),
             "gamma": (1.0 + 0.2 * torch.randn(c, generator=gen, device=dev)).to(params),
             "beta": (0.2 * torch.randn(c, generator=gen, device=dev)).to(params)}
    if case["op"] == "norm_grad":
        state["dy"] = _channels_last(torch.randn(stored, generator=gen, device=dev).to(dtype))
        # the forward pass left its statistics
        state["mean"], state["rstd"] = _plain_statistics(state["x"], case["groups"], 1e-5)
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    state = {"case": case, "seed": seed * 0x9E3779B97F4A7C15 & 0xFFFFFFFFFFFFFFFF, "offset": 3}
    if case["op"] in ("norm", "norm_grad"):
        state.update(_norm_state(case, seed, gen, dev))
    elif case["op"] == "dropout":
        state["x"] = torch.randn(case["count"], generator=gen, device=dev).to(dtype)
        if case["residual"]:
            state["residual"] = torch.randn(case["count"], generator=gen, device=dev).to(dtype)
    else:
        # tokens by their rank of use: the k-th most used in proportion to 1 / k, names shuffled
        u = torch.rand(case["tokens"], generator=gen, device=dev, dtype=torch.float64)
        rank = (torch.exp(u * math.log(case["rows"] + 1)).long() - 1).clamp_(0, case["rows"] - 1)
        ids = torch.randperm(case["rows"], generator=gen, device=dev)[rank]
        if case["padding"]:  # the shorter texts of a batch end in padding
            ids[torch.rand(case["tokens"], generator=gen, device=dev) < 0.3] = 0
        state["ids"] = ids.to(torch.int64 if case["ids"] == "int64" else torch.int32)
        state["scale"] = math.sqrt(case["width"])
        if case["op"] == "embed":
            state["table"] = torch.randn((case["rows"], case["width"]), generator=gen, device=dev).to(dtype)
        else:
            state["dy"] = torch.randn((case["tokens"], case["width"]), generator=gen, device=dev).to(dtype)
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
    random = dict(seed=state["seed"], offset=state["offset"])
    if case["op"] == "norm":
        return T.PreparedCall(T.group_norm_nd, state["x"], case["groups"], state["gamma"], state["beta"], eps=1e-5,
                              activation=case["act"], dropout_p=case["p"], **random)
    if case["op"] == "norm_grad":
        return T.PreparedCall(T.group_norm_backward_nd, state["dy"], state["x"], state["mean"], state["rstd"],
                              case["groups"], state["gamma"], state["beta"], activation=case["act"],
                              dropout_p=case["p"], **random)
    if case["op"] == "dropout":
        return T.PreparedCall(T.dropout_nd, state["x"], case["p"], residual=state.get("residual"), **random)
    if case["op"] == "embed":
        return T.PreparedCall(T.embedding_nd, state["ids"], state["table"], scale=state["scale"])
    return T.PreparedCall(T.embedding_backward_nd, state["dy"], state["ids"], case["rows"], scale=state["scale"],
                          padding_idx=0 if case["padding"] else None)


def run(state):
    if own:
        return state["call"]()
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dropout": _plain_dropout, "embed": _plain_embed,
            "embed_grad": _plain_embed_grad}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------
# the plain forms: elementary torch operations in 32 bits, rounded once at the end
# ------------------------------------------------------------------------------------
def _grouped(x, groups):
    """(N, C, D..) stored channels last, as (N, P, G, C/G) in 32 bits."""
    return x.movedim(1, -1).reshape(x.shape[0], -1, groups, x.shape[1] // groups).float()


def _plain_statistics(x, groups, eps):
    v = _grouped(x, groups)
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return mean, 1.0 / torch.sqrt(var + eps)


def _round(words, key):
    """One round of the Philox 4x32 generator (Salmon et al. 2011) on 32-bit words held in int64."""
    c0, c1, c2, c3 = words
    p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return ((p1 >> 32 & MASK32) ^ c1 ^ key[0], p1 & MASK32, (p0 >> 32 & MASK32) ^ c3 ^ key[1], p0 & MASK32)


def _plain_keep(count, p, seed, offset, dev):
    """Which of `count` elements stay: eight 16-bit fields of each counter, against p in 1 / 65536."""
    i = torch.arange((count + 7) // 8, device=dev)
    low, high = offset & MASK32, offset >> 32 & MASK32
    keys = [((seed + r * 0x9E3779B9) & MASK32, ((seed >> 32) + r * 0xBB67AE85) & MASK32) for r in range(10)]
    words = (i & MASK32, i >> 32, torch.full_like(i, low), torch.full_like(i, high))
    words = torch.stack(functools.reduce(_round, keys, words), 1)
    fields = torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:count]
    return fields >= _threshold(p)


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _factor(p):
    return 65536.0 / (65536 - _threshold(p))


def _plain_drop(v, p, state):
    """Dropout of `v`, its elements numbered in storage order."""
    if not p:
        return v
    keep = _plain_keep(v.numel(), p, state["seed"], state["offset"], v.device).reshape(v.shape)
    return torch.where(keep, v * _factor(p), 0.0)


def _activation(z, kind):
    return {"silu": lambda: z / (1.0 + torch.exp(-z)), "identity": lambda: z, "relu": lambda: z.clamp(min=0.0)}[kind]()


def _ungrouped(v, like):
    """(N, P, G, C/G) in 32 bits, as a tensor of `like`'s type and channels-last shape."""
    return _channels_last(v.to(like.dtype).reshape(like.movedim(1, -1).shape))


def _plain_norm(state):
    case, x = state["case"], state["x"]
    mean, rstd = _plain_statistics(x, case["groups"], 1e-5)
    xhat = (_grouped(x, case["groups"]) - mean[:, None, :, None]) * rstd[:, None, :, None]
    gamma, beta = (state[k].float().reshape(case["groups"], -1) for k in ("gamma", "beta"))
    y = _plain_drop(_activation(xhat * gamma + beta, case["act"]), case["p"], state)
    return _ungrouped(y, x), mean, rstd


def _plain_norm_grad(state):
    case, x, groups = state["case"], state["x"], state["case"]["groups"]
    mean, rstd = (state[k][:, None, :, None] for k in ("mean", "rstd"))
    gamma, beta = (state[k].float().reshape(groups, -1) for k in ("gamma", "beta"))
    xhat = (_grouped(x, groups) - mean) * rstd
    dz = _plain_drop(_grouped(state["dy"], groups), case["p"], state)
    if case["act"] == "silu":
        z = xhat * gamma + beta
        s = 1.0 / (1.0 + torch.exp(-z))
        dz = dz * (s * (1.0 + z * (1.0 - s)))
    dgamma, dbeta = (dz * xhat).sum((0, 1)).reshape(-1), dz.sum((0, 1)).reshape(-1)
    g = dz * gamma
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - xhat * (g * xhat).mean((1, 3), keepdim=True))
    return _ungrouped(dx, x), dgamma.to(state["gamma"].dtype), dbeta.to(state["beta"].dtype)


def _plain_dropout(state):
    y = _plain_drop(state["x"].float(), state["case"]["p"], state)
    return (y + state["residual"].float() if "residual" in state else y).to(state["x"].dtype)


def _plain_embed(state):
    return (state["table"][state["ids"].long()].float() * state["scale"]).to(state["table"].dtype)


def _plain_embed_grad(state):
    case, ids = state["case"], state["ids"].long()
    dy = state["dy"].float() * state["scale"]
    if case["padding"]:
        dy = torch.where((ids == 0)[:, None], 0.0, dy)
    total = torch.zeros((case["rows"], case["width"]), device=dy.device).index_add_(0, ids, dy)
    return total.to(state["dy"].dtype)


# ------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------
def _exact_keep(count, p, seed, offset):
    """The same generator written on numpy's unsigned words."""
    n, m = (count + 7) // 8, np.uint64(MASK32)
    i = np.arange(n, dtype=np.uint64)
    a, b = i & m, i >> np.uint64(32)
    c, d = np.full(n, offset & MASK32, np.uint64), np.full(n, offset >> 32, np.uint64)
    k0, k1 = seed & MASK32, seed >> 32
    for _ in range(10):
        e, f = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (f >> np.uint64(32)) ^ b ^ np.uint64(k0), f & m, (e >> np.uint64(32)) ^ d ^ np.uint64(k1), e & m
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    fields = np.stack([a, b, c, d], 1).astype("<u4").view("<u2").reshape(-1)[:count]
    return torch.from_numpy(fields.astype(np.int32) >= int(p * 65536 + 0.5))


def _exact_drop(v, state):
    p = state["case"]["p"]
    if p == 0.0:
        return v
    keep = _exact_keep(v.numel(), p, state["seed"], state["offset"]).to(v.device).reshape(v.shape)
    return v * keep * (65536.0 / (65536.0 - int(p * 65536 + 0.5)))


def _exact_norm(state):
    case, x = state["case"], state["x"].double()
    n, c = x.shape[:2]
    by_group = (n, case["groups"], c // case["groups"], -1)
    v = x.reshape(by_group)
    var, mean = torch.var_mean(v, (2, 3), correction=0)
    z = (v - mean[..., None, None]) * (var + 1e-5).rsqrt()[..., None, None]
    per_channel = (1, case["groups"], c // case["groups"], 1)
    z = z * state["gamma"].double().reshape(per_channel) + state["beta"].double().reshape(per_channel)
    z = {"silu": lambda: z * torch.sigmoid(z), "identity": lambda: z, "relu": lambda: torch.relu(z)}[case["act"]]()
    y = _exact_drop(z.reshape(x.shape).movedim(1, -1).contiguous(), state).movedim(-1, 1)
    return y, mean, (var + 1e-5).rsqrt()


def _exact_norm_grad(state):
    case = state["case"]
    x, n, c = state["x"].double(), case["n"], case["c"]
    cg = c // case["groups"]
    e = _exact_drop(state["dy"].double().movedim(1, -1).contiguous(), state).movedim(-1, 1).reshape(n, c, -1)
    wide = lambda t: t.double().repeat_interleave(cg, 1)[:, :, None]  # noqa: E731
    rstd, gamma = wide(state["rstd"]), state["gamma"].double()[None, :, None]
    xhat = (x.reshape(n, c, -1) - wide(state["mean"])) * rstd
    if case["act"] == "silu":
        z = xhat * gamma + state["beta"].double()[None, :, None]
        s = torch.sigmoid(z)
        e = e * (s + z * s * (1.0 - s))
    count = cg * e.shape[2]
    c1 = (e * gamma).sum(2).reshape(n, -1, cg).sum(2) / count
    c2 = (e * gamma * xhat).sum(2).reshape(n, -1, cg).sum(2) / count
    dx = rstd * (e * gamma - wide(c1) - xhat * wide(c2))
    return dx.reshape(x.shape), (e * xhat).sum((0, 2)), e.sum((0, 2))


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(state)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(state)
    if case["op"] == "dropout":
        y = _exact_drop(state["x"].double(), state)
        return y + state["residual"].double() if case["residual"] else y
    ids = state["ids"].long()
    if case["op"] == "embed":
        return torch.index_select(state["table"].double(), 0, ids) * state["scale"]
    kept = ids != 0 if case["padding"] else torch.ones_like(ids, dtype=torch.bool)
    table = torch.zeros((case["rows"], case["width"]), dtype=torch.float64, device=ids.device)
    table.index_put_((ids[kept],), state["dy"].double()[kept], accumulate=True)
    return table * state["scale"]


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        count = math.prod(_shape(case))
        params, stats = 2 * case["c"] * SIZE[case["params"]], 2 * 4 * case["n"] * case["groups"]
        if case["op"] == "norm":
            return {"bytes": 2 * count * size + params + stats, "flops": 12 * count}
        return {"bytes": 3 * count * size + 2 * params + stats, "flops": 25 * count}
    if case["op"] == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * case["count"] * size, "flops": 2 * case["count"]}
    ids = case["tokens"] * (8 if case["ids"] == "int64" else 4)
    moved = case["tokens"] * case["width"] * size
    if case["op"] == "embed":  # the distinct rows that this use of codes reads, about
        k = case["rows"]
        share = case["tokens"] / math.log(k + 1)
        distinct = min(k, case["tokens"], share * (1 + math.log(max(1.0, k / max(share, 1.0)))) if share < k else k)
        return {"bytes": ids + moved + int(distinct) * case["width"] * size, "flops": case["tokens"] * case["width"]}
    return {"bytes": ids + moved + case["rows"] * case["width"] * size, "flops": case["tokens"] * case["width"]}
