"""Cases of the operators around one fine-tuning step of a quantized
feed-forward block: adapters with dropout, the gated block, and the
likelihood that the step trains.

Five operators, each in its plain form (elementary torch operations in 32 bits)
and through the package:

  linear     Y = X.W^T + s (D(X).A^T).B^T, D the dropout of the adapter's input;
  backward   its gradients dX, dA and dB;
  gated      H = act(G) * U with G and U two such layers of one X (one D(X) for
             both), G and U themselves (what the backward pass needs) and the
             low-rank factors;
  gradients  its gradients: dX and dA, dB of both layers;
  logprobs   log-probabilities of given tokens, entropies, the k most likely
             tokens, and their gradient.

D keeps element i of X where the i % 8 th 16-bit piece of the counter-based
generator's 128 bits for i / 8 is at least round(65536 p), times what that
leaves of 1; the mask is a function of (seed, offset, i) and is stored nowhere.

The weights are stored as 4-bit codes of 64-element blocks with doubly
quantized constants (the library's format); their dequantized values, rounded
to bf16, are what the layers are defined on.
"""

import math

import numpy as np
import torch

own = False

# the 16 levels of the 4-bit code, as fp32
LEVELS = (-1.0, -0.6934942007064819, -0.5225629806518555, -0.39286819100379944, -0.282901793718338,
          -0.183749720454216, -0.09053941816091537, 0.0, 0.07913367450237274, 0.16003505885601044,
          0.2447662651538849, 0.3361186981201172, 0.43847718834877014, 0.5600152611732483, 0.7202957272529602, 1.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # the tokens of a small evaluation during training, dropout still on
        {"name": "linear-few", "op": "linear", "m": 9, "n": 4096, "k": 4096, "r": 16, "p": 0.05, "out": "bf16"},
        # a training batch through the gate projection
        {"name": "linear-batch", "op": "linear", "m": 4096, "n": 11008, "k": 4096, "r": 64, "p": 0.1, "out": "bf16"},
        # a short sequence in training, the low-rank factor not kept, fp32 gradient
        {"name": "backward-short", "op": "backward", "m": 61, "n": 4096, "k": 4096, "r": 8, "p": 0.1, "out": "f32",
         "saved": False},
        # a training batch through the down projection
        {"name": "backward-batch", "op": "backward", "m": 4096, "n": 4096, "k": 11008, "r": 64, "p": 0.05,
         "out": "bf16", "saved": True},
        # the next token of one user
        {"name": "gated-token", "op": "gated", "m": 1, "n": 11008, "k": 4096, "r": 16, "p": 0.0, "act": "silu",
         "save": False},
        # the next tokens of an odd number of users
        {"name": "gated-13-tokens", "op": "gated", "m": 13, "n": 11008, "k": 4096, "r": 64, "p": 0.0, "act": "silu",
         "save": False},
        # a training batch
        {"name": "gated-batch", "op": "gated", "m": 4096, "n": 11008, "k": 4096, "r": 64, "p": 0.1, "act": "silu",
         "save": True},
        # an odd number of tokens, the other activation
        {"name": "gradients-odd", "op": "gradients", "m": 509, "n": 5504, "k": 2048, "r": 16, "p": 0.05,
         "act": "gelu_tanh", "out": "bf16", "saved": False},
        # a training batch
        {"name": "gradients-batch", "op": "gradients", "m": 4096, "n": 11008, "k": 4096, "r": 64, "p": 0.1,
         "act": "silu", "out": "bf16", "saved": True},
        # what a server reports beside its tokens
        {"name": "logprobs-served", "op": "logprobs", "m": 32, "v": 32000, "ld": 32000, "top": 20, "tau": 1.0,
         "z": "bf16", "part": "score", "masked": 0.0},
        # the loss and the gradient of a training batch
        {"name": "logprobs-batch", "op": "logprobs", "m": 4096, "v": 32000, "ld": 32000, "top": 0, "tau": 1.0,
         "z": "bf16", "part": "train", "masked": 0.0},
        # the gradient of likelihood and entropy from what the first pass kept: odd vocabulary in padded rows, fp32
        {"name": "logprobs-gradient", "op": "logprobs", "m": 777, "v": 50001, "ld": 50008, "top": 0, "tau": 1.5,
         "z": "f32", "part": "gradient", "masked": 0.1},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "backward", "gated", "gradients", "logprobs", "logprobs"))
    if op == "logprobs":
        v = _log_int(rng, 1000, 130000)
        m = min(_log_int(rng, 1, 4096), max(1, 4096 * 32000 // v))
        part = rng.choice(("score", "train", "gradient"))
        return {"op": op, "m": m, "v": v, "ld": -(-v // 8) * 8 + rng.choice((0, 0, 56)),
                "top": _log_int(rng, 1, 64) if part == "score" else 0, "tau": rng.choice((0.7, 1.0, 1.0, 2.0)),
                "z": rng.choice(("bf16", "bf16", "f16", "f32")), "part": part, "masked": rng.choice((0.0, 0.0, 0.3))}
    while True:
        m, n, k = _log_int(rng, 1, 4096), 8 * _log_int(rng, 64, 1376), 64 * _log_int(rng, 8, 172)
        if m * n * k <= 4096 * 11008 * 4096:
            break
    case = {"op": op, "m": m, "n": n, "k": k, "r": 8 * _log_int(rng, 1, 16), "p": rng.choice((0.0, 0.05, 0.1, 0.3))}
    if op in ("gated", "gradients"):
        case["act"] = rng.choice(("silu", "silu", "gelu_tanh"))
    if op == "gated":
        case["save"] = rng.choice((True, False))
    else:
        case["out"] = rng.choice(("bf16", "bf16", "f32"))
    if op in ("backward", "gradients"):
        case["saved"] = rng.choice((True, False))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _quantized(gen, n, k):
    """A frozen weight N(0, 0.02^2) in the library's 4-bit format."""
    dev = torch.device("cuda")
    w = torch.randn(n * k // 64, 64, generator=gen, device=dev) * 0.02
    c = w.abs().amax(1)
    levels = torch.tensor(LEVELS, device=dev)
    code = torch.bucketize(w / c[:, None], (levels[1:] + levels[:-1]) / 2).to(torch.uint8).view(-1, 2)
    codes = code[:, 0] | (code[:, 1] << 4)
    mean = c.double().mean().float().view(1)
    d = c - mean
    blocks = d.numel()
    groups = -(-blocks // 256)
    padded = torch.zeros(groups * 256, device=dev)
    padded[:blocks] = d
    scale = padded.view(groups, 256).abs().amax(1) / 448
    const = (padded.view(groups, 256) / scale.clamp_min(1e-30)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    const = const.view(torch.uint8).view(-1)[:blocks].contiguous()
    return {"codes": codes.contiguous(), "const": const, "scale": scale, "mean": mean}


ALPHA = 16.0


def _layers(case):
    return 2 if case["op"] in ("gated", "gradients") else 1


def _layer_inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 2 + 1)
    m, n, k, r = (case[x] for x in ("m", "n", "k", "r"))

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(torch.bfloat16)

    state = {"case": case, "x": normal(m, k), "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 63, "offset": seed % 1000,
             "w": [_quantized(gen, n, k) for _ in range(_layers(case))],
             "a": [normal(r, k, scale=0.02) for _ in range(_layers(case))],
             "b": [normal(n, r, scale=0.02) for _ in range(_layers(case))]}
    if case["op"] == "backward":
        state["dy"] = normal(m, n)
    if case["op"] == "gradients":
        state["dh"] = normal(m, n)
        # what the forward pass kept: X.W^T spreads as sqrt(k) times the weight
        state["g"] = normal(m, n, scale=0.02 * math.sqrt(k))
        state["u"] = normal(m, n, scale=0.02 * math.sqrt(k))
    if case.get("saved"):
        x = torch.where(_kept(state), state["x"].float(), 0.0)
        state["t"] = torch.stack([(x @ a.float().T) * _kept_scale(case) for a in state["a"]])
    else:
        state["t"] = None
    return state


def _logprobs_inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 2 + 1)
    m, v, ld = case["m"], case["v"], case["ld"]
    z = torch.randn(m, ld, generator=gen, device=dev) * 2.5
    # the given token is often a likely one
    likely = z[:, :v].argmax(1)
    target = torch.where(torch.rand(m, generator=gen, device=dev) < 0.4, likely,
                         torch.randint(0, v, (m,), generator=gen, device=dev))
    # tokens that sampling rules out
    if case["masked"]:
        out = torch.rand(m, v, generator=gen, device=dev) < case["masked"]
        out.scatter_(1, target[:, None], False)
        z[:, :v].masked_fill_(out, -math.inf)
    # prompt and padding carry no target
    target = torch.where(torch.rand(m, generator=gen, device=dev) < 0.1, -100, target)
    up = 1024.0 if case["z"] == "f16" else 1.0
    state = {"case": case, "z": z.to(DTYPES[case["z"]]), "target": target.to(torch.int32),
             "dlogp": -up * (torch.rand(m, generator=gen, device=dev) + 0.5) / m,
             "dentropy": None}
    if case["part"] == "gradient":
        state["dentropy"] = up * 0.02 * torch.rand(m, generator=gen, device=dev) / m
        x = state["z"][:, :v].double() / case["tau"]
        lse = torch.logsumexp(x, 1)
        log_q = x - lse[:, None]
        state["lse"] = lse.float()
        state["entropy"] = -torch.where(log_q > -1e30, log_q.exp() * log_q, 0.0).sum(1).float()
    return state


def prepare(case, seed):
    state = _logprobs_inputs(case, seed) if case["op"] == "logprobs" else _layer_inputs(case, seed)
    if not own:
        return state
    import quantized_fine_tuning_amd as q

    dev, m = "cuda", case["m"]
    if case["op"] == "logprobs":
        if case["part"] != "gradient":
            state["logp"], state["lse_out"] = torch.empty(m, device=dev), torch.empty(m, device=dev)
            state["entropy_out"] = torch.empty(m, device=dev) if case["part"] == "score" else None
        if case["part"] != "score":
            state["dz"] = torch.empty_like(state["z"])
        state["top_logp"] = torch.empty(m, case["top"], device=dev) if case["top"] else None
        state["top_index"] = torch.empty(m, case["top"], dtype=torch.int32, device=dev) if case["top"] else None
        return state
    n, k, r = case["n"], case["k"], case["r"]
    state["weight"] = [q.Nf4Tensor(n, k, w["codes"], w["const"], w["scale"], w["mean"]) for w in state["w"]]
    state["drop"] = q.Dropout(case["p"], state["seed"], state["offset"]) if case["p"] else None
    forward = case["op"] in ("linear", "gated")
    sizes = (q.qlora_gated_sizes if _layers(case) == 2 else q.qlora_dropout_linear_sizes)(n, k, m, r)
    state["ws"] = q.workspace(sizes["fwd_ws_bytes" if forward else "bwd_ws_bytes"])
    if case["op"] == "linear":
        state["y"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device=dev)
        state["t_out"] = torch.empty(m, r, device=dev)
    elif case["op"] == "gated":
        state["h"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
        keep = case["save"]
        state["g_out"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev) if keep else None
        state["u_out"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev) if keep else None
        state["t_out"] = torch.empty(2, m, r, device=dev) if keep else None
    else:
        state["dx"] = torch.empty(m, k, dtype=DTYPES[case["out"]], device=dev)
        state["da"] = [torch.empty(r, k, device=dev) for _ in state["w"]]
        state["db"] = [torch.empty(n, r, device=dev) for _ in state["w"]]
    if _layers(case) == 2:
        state["adapters"] = q.GatedAdapters(state["a"][0], state["b"][0], state["a"][1], state["b"][1], ALPHA)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _weight(w, n, k):
    """The dequantized weight: RNE_bf16(level[code] * (e4m3 * scale + mean))."""
    codes = w["codes"].to(torch.int32)
    levels = torch.tensor(LEVELS, device=codes.device)
    value = torch.stack((levels[codes & 15], levels[codes >> 4]), 1).view(-1, 64)
    group = torch.arange(value.shape[0], device=codes.device) // 256
    const = w["const"].view(torch.float8_e4m3fn).float() * w["scale"][group] + w["mean"]
    return (value * const[:, None]).to(torch.bfloat16).float().view(n, k)


def _threshold(case):
    return int(round(case["p"] * 65536))


def _kept_scale(case):
    return 65536.0 / (65536 - _threshold(case))


def _kept(state):
    """Which elements of X are kept: ten rounds of the 4x32-bit counter-based generator (Salmon, Moraes, Dror and
    Shaw 2011) under the 64-bit key `seed`, the counter (i / 8, offset)."""
    m, k = state["x"].shape
    low = 0xFFFFFFFF
    i = torch.arange(m * k // 8, device=state["x"].device)
    c0, c1 = i & low, i >> 32
    c2, c3 = torch.full_like(i, state["offset"] & low), torch.full_like(i, state["offset"] >> 32)
    k0, k1 = state["seed"] & low, state["seed"] >> 32
    for _ in range(10):
        # (the products pass 2^63 and wrap: their bits are the 64-bit products' all the same)
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), 1)
    pieces = torch.stack((words & 0xFFFF, words >> 16), 2)
    return pieces.view(m, k) >= _threshold(state["case"])


def _gate(act, g):
    """(act(g) / g, act'(g))"""
    if act == "silu":
        s = torch.sigmoid(g)
        return s, s * (1 + g * (1 - s))
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g * g * g))
    return s, s * (1 + g * (1 - s) * (c * (1 + 3 * 0.044715 * g * g)))


def _plain_layers(state):
    """(X, D(X), weights, s) in 32 bits."""
    case = state["case"]
    x = state["x"].float()
    dropped = torch.where(_kept(state), x, 0.0) * _kept_scale(case) if case["p"] else x
    return x, dropped, [_weight(w, case["n"], case["k"]) for w in state["w"]], ALPHA / case["r"]


def _plain_forward(state):
    case = state["case"]
    x, dropped, weights, s = _plain_layers(state)
    t = [dropped @ a.float().T for a in state["a"]]
    y = [x @ w.T + s * (f @ b.float().T) for w, f, b in zip(weights, t, state["b"])]
    if case["op"] == "linear":
        return {"y": y[0].to(DTYPES[case["out"]]), "t": t[0]}
    out = {"h": (y[0] * _gate(case["act"], y[0])[0] * y[1]).to(torch.bfloat16)}
    if case["save"]:
        out |= {"g": y[0].to(torch.bfloat16), "u": y[1].to(torch.bfloat16), "t": torch.stack(t)}
    return out


def _plain_gradients(state):
    """The outgoing gradients of the layers, in their 16 bits (in 64 on the way there: the next products take them as
    they are rounded, and 32 bits fall on the other side of a border now and then)."""
    if state["case"]["op"] == "backward":
        return [state["dy"].float()]
    dh, g, u = state["dh"].double(), state["g"].double(), state["u"].double()
    share, slope = _gate(state["case"]["act"], g)
    return [(dh * u * slope).to(torch.bfloat16).float(), (dh * (g * share)).to(torch.bfloat16).float()]


def _plain_backward(state):
    case = state["case"]
    _, dropped, weights, s = _plain_layers(state)
    dy = _plain_gradients(state)
    t = [dropped @ a.float().T for a in state["a"]] if state["t"] is None else list(state["t"])
    u = [s * (d @ b.float()) for d, b in zip(dy, state["b"])]
    low = sum(f @ a.float() for f, a in zip(u, state["a"]))
    if case["p"]:
        low = torch.where(_kept(state), low, 0.0) * _kept_scale(case)
    dx = sum(d @ w for d, w in zip(dy, weights)) + low
    return {"dx": dx.to(DTYPES[case["out"]]), "da": [f.T @ dropped for f in u],
            "db": [s * (d.T @ f) for d, f in zip(dy, t)]}


def _plain_logprobs(state):
    case = state["case"]
    v, tau, part = case["v"], case["tau"], case["part"]
    z = state["z"][:, :v].float() / tau
    has = (state["target"] >= 0) & (state["target"] < v)
    at = torch.where(has, state["target"], 0).long()[:, None]
    out = {}
    if part == "gradient":
        lse, entropy = state["lse"], state["entropy"]
    else:
        high = z.amax(1, keepdim=True)
        e = torch.exp(z - high)
        total = e.sum(1)
        lse = high[:, 0] + torch.log(total)
        # against the row's largest: both logarithms are near their size, not the logits'
        out = {"logp": torch.where(has, (z.gather(1, at) - high)[:, 0] - torch.log(total), 0.0), "lse": lse}
        if part == "score":
            out["entropy"] = torch.log(total) - torch.where(e > 0, (z - high) * e, 0.0).sum(1) / total
            # equal logits by their index
            value, index = torch.sort(state["z"][:, :v], dim=1, descending=True, stable=True)
            out["top_logp"] = value[:, :case["top"]].float() / tau - lse[:, None]
            out["top_index"] = index[:, :case["top"]].to(torch.int32)
            return out
    log_q = z - lse[:, None]
    q = torch.exp(log_q)
    dlogp = torch.where(has, state["dlogp"], 0.0)
    dz = -dlogp[:, None] * q
    dz.scatter_add_(1, at, dlogp[:, None])
    if state["dentropy"] is not None:
        dz -= state["dentropy"][:, None] * torch.where(q > 0, q * (log_q + entropy[:, None]), 0.0)
    out["dz"] = torch.zeros_like(state["z"])
    out["dz"][:, :v] = (dz / tau).to(out["dz"].dtype)
    return out


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "logprobs":
            return _plain_logprobs(state)
        return _plain_forward(state) if case["op"] in ("linear", "gated") else _plain_backward(state)
    import quantized_fine_tuning_amd as q

    if case["op"] == "logprobs":
        if case["part"] == "gradient":
            q.qlora_logprobs_bwd(state["z"], state["target"], case["tau"], state["lse"], state["dlogp"], state["dz"],
                                 entropy=state["entropy"], d_entropy=state["dentropy"], vocab=case["v"])
            return {"dz": state["dz"]}
        train = case["part"] == "train"
        q.qlora_logprobs_fwd(state["z"], state["target"], case["tau"], state["logp"], state["lse_out"],
                             entropy=state["entropy_out"], top_logp=state["top_logp"], top_index=state["top_index"],
                             d_logp=state["dlogp"] if train else None, dZ=state["dz"] if train else None,
                             vocab=case["v"])
        out = {"logp": state["logp"], "lse": state["lse_out"]}
        if train:
            return out | {"dz": state["dz"]}
        return out | {"entropy": state["entropy_out"], "top_logp": state["top_logp"], "top_index": state["top_index"]}
    if case["op"] == "linear":
        q.qlora_dropout_linear_fwd(state["weight"][0], state["x"], state["a"][0], state["b"][0], case["r"], ALPHA,
                                   state["drop"], state["y"], state["t_out"], state["ws"])
        return {"y": state["y"], "t": state["t_out"]}
    if case["op"] == "gated":
        q.qlora_gated_fwd(state["weight"][0], state["weight"][1], state["x"], state["adapters"], case["act"],
                          state["drop"], state["h"], state["g_out"], state["u_out"], state["t_out"], state["ws"])
        out = {"h": state["h"]}
        if case["save"]:
            out |= {"g": state["g_out"], "u": state["u_out"], "t": state["t_out"]}
        return out
    if case["op"] == "backward":
        q.qlora_dropout_linear_bwd(state["weight"][0], state["x"], state["dy"], state["a"][0], state["b"][0],
                                   case["r"], ALPHA, state["drop"], None if state["t"] is None else state["t"][0],
                                   state["dx"], state["da"][0], state["db"][0], state["ws"])
    else:
        q.qlora_gated_bwd(state["weight"][0], state["weight"][1], state["x"], state["dh"], state["g"], state["u"],
                          state["adapters"], case["act"], state["drop"], state["t"], state["dx"], state["da"][0],
                          state["db"][0], state["da"][1], state["db"][1], state["ws"])
    return {"dx": state["dx"], "da": state["da"], "db": state["db"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact result
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "logprobs":
        m, v, size = case["m"], case["v"], SIZES[case["z"]]
        gradient = 0 if case["part"] == "score" else m * case["ld"] * size
        return {"bytes": m * v * size + gradient + 8 * m * case["top"] + 20 * m,
                "flops": m * v * (6 if case["part"] == "score" else 8)}
    m, n, k, r = (case[x] for x in ("m", "n", "k", "r"))
    layers = _layers(case)
    weight = n * k // 2 + n * k // 64 + n * k // 64 // 256 * 4 + 2 * r * (n + k)
    if case["op"] == "linear":
        moved = 2 * m * k + SIZES[case["out"]] * m * n + 4 * m * r
    elif case["op"] == "gated":
        moved = 2 * m * k + 2 * m * n + (4 * m * n + 8 * m * r if case["save"] else 0)
    else:
        moved = 2 * m * k + (2 if layers == 1 else 6) * m * n + SIZES[case["out"]] * m * k
        moved += layers * (4 * r * (n + k) + (4 * m * r if case["saved"] else 0))
    low = 2 * m * r * (n + k)
    if case["op"] in ("backward", "gradients"):
        low = 2 * m * r * (2 * n + 2 * k + (0 if case["saved"] else k))
    return {"bytes": layers * weight + moved, "flops": layers * (2 * m * n * k + low)}


def _exact_weight(w, n, k):
    # every step of the definition is a rounding to 32 or 16 bits, so it is made in those
    byte = w["const"].to(torch.int64)
    sign = 1.0 - 2.0 * (byte >> 7).double()
    power, mantissa = (byte >> 3) & 15, (byte & 7).double()
    value = torch.where(power > 0, (1 + mantissa / 8) * torch.exp2(power.double() - 7), mantissa * 2.0 ** -9) * sign
    scale = w["scale"].double().repeat_interleave(256)[:byte.numel()]
    const = ((value * scale).float().double() + w["mean"].double()).float().double()
    level = torch.tensor(LEVELS, device=byte.device, dtype=torch.float64)
    codes = w["codes"].view(-1, 32).to(torch.int64)
    out = torch.empty(byte.numel(), 64, dtype=torch.float64, device=byte.device)
    out[:, 0::2] = level[codes % 16]
    out[:, 1::2] = level[codes // 16]
    return (out * const[:, None]).float().to(torch.bfloat16).double().view(n, k)


def _exact_dropout(case, s):
    """What X is multiplied with, element by element, from the generator in unsigned host arithmetic."""
    if not case["p"]:
        return 1.0
    n = case["m"] * case["k"] // 8
    mask, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [np.arange(n, dtype=np.uint64), np.zeros(n, np.uint64), np.full(n, s["offset"], np.uint64), np.zeros(n, np.uint64)]
    key = np.array([s["seed"] % 2 ** 32, s["seed"] // 2 ** 32], dtype=np.uint64)
    for _ in range(10):
        p, q = x[0] * np.uint64(3528531795), x[2] * np.uint64(3449720151)
        x = [(q >> shift) ^ x[1] ^ key[0], q & mask, (p >> shift) ^ x[3] ^ key[1], p & mask]
        key = (key + np.array([2654435769, 3144134277], dtype=np.uint64)) & mask
    bits = np.stack(x, 1).astype("<u4").view("<u2").reshape(case["m"], case["k"])
    out = int(round(case["p"] * 65536))
    keep = torch.from_numpy((bits >= out).astype(np.float64)).to(s["x"].device)
    return keep * (65536 / (65536 - out))


def _exact_act(act, g):
    """act(g) and its derivative, through tanh."""
    if act == "silu":
        half = torch.tanh(g / 2)
        return g * (1 + half) / 2, (1 + half) / 2 + g * (1 - half * half) / 4
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * c * (1 + 0.134145 * g ** 2)


def _exact_logprobs(case, seed):
    s = _logprobs_inputs(case, seed)
    v, tau, m = case["v"], case["tau"], case["m"]
    z = s["z"].double()[:, :v] / tau
    log_q = torch.log_softmax(z, 1)
    line = torch.arange(m, device=z.device)
    known = (s["target"] >= 0).nonzero()[:, 0]
    column = s["target"].long()[known]
    if case["part"] == "gradient":
        log_q = z - s["lse"].double()[:, None]
    q = log_q.exp()
    got = {}
    if case["part"] != "gradient":
        logp = torch.zeros(m, dtype=torch.float64, device=z.device)
        logp[known] = log_q[known, column]
        got = {"logp": logp, "lse": torch.logsumexp(z, 1)}
    if case["part"] == "score":
        got["entropy"] = torch.special.entr(q).sum(1)
        got["top_logp"] = log_q.topk(case["top"], 1).values
        got["top_index"] = None
        return got
    dz = torch.zeros(m, case["ld"], dtype=torch.float64, device=z.device)
    weight = torch.zeros(m, dtype=torch.float64, device=z.device)
    weight[known] = s["dlogp"].double()[known]
    dz[:, :v] = -q * weight[:, None]
    dz[line[known], column] += weight[known]
    if s["dentropy"] is not None:
        part = torch.special.entr(q) - q * s["entropy"].double()[:, None]
        dz[:, :v] += s["dentropy"].double()[:, None] * part
    got["dz"] = dz / tau
    return got


def exact(case, seed):
    if case["op"] == "logprobs":
        return _exact_logprobs(case, seed)
    s = _layer_inputs(case, seed)
    x, scale = s["x"].double(), ALPHA / case["r"]
    factor = _exact_dropout(case, s)
    a, b = [v.double() for v in s["a"]], [v.double() for v in s["b"]]
    if s["t"] is None:
        t = [torch.mm(x * factor, v.t()) for v in a]
    else:
        t = [v.double() for v in s["t"]]
    if case["op"] in ("linear", "gated"):
        y = [torch.addmm(torch.mm(x, _exact_weight(w, case["n"], case["k"]).t()), f, v.t(), alpha=scale)
             for w, f, v in zip(s["w"], t, b)]
        if case["op"] == "linear":
            return {"y": y[0], "t": t[0]}
        got = {"h": _exact_act(case["act"], y[0])[0] * y[1]}
        if case["save"]:
            got |= {"g": y[0], "u": y[1], "t": torch.stack(t)}
        return got
    if case["op"] == "backward":
        dy = [s["dy"].double()]
    else:
        # the definition rounds what reaches the two layers to their 16 bits
        value, slope = _exact_act(case["act"], s["g"].double())
        dh = s["dh"].double()
        dy = [(slope * s["u"].double() * dh).to(torch.bfloat16).double(), (value * dh).to(torch.bfloat16).double()]
    dx = torch.zeros_like(x)
    got = {"da": [], "db": []}
    for i, d in enumerate(dy):
        u = scale * torch.mm(d, b[i])
        dx += torch.mm(d, _exact_weight(s["w"][i], case["n"], case["k"])) + torch.mm(u, a[i]) * factor
        got["da"].append(torch.mm(u.t(), x * factor))
        got["db"].append(scale * torch.mm(d.t(), t[i]))
    return got | {"dx": dx}
