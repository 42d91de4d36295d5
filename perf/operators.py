"""The operators of a recurrent language-model block, as cases to be measured.

  prompt    linear attention with a decay for each head over whole (packed) sequences
  train     the same with its gradients
  step      its recurrent form: one token for every sequence of a batch
  addnorm   residual add with a scale, and the norm in front of a block
  gatenorm  the gated norm behind a block's mixer, by groups of channels

Where ``own`` is false, ``run`` computes them in elementary torch operations
in 32 bits; where it is true it calls the package.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few short requests prefilled together from cached states, one of
        # them a single token and one empty: latency counts
        {"name": "prompt_ragged_bf16", "op": "prompt", "lens": "1,37,64,130,0,411", "H": 16,
         "G": 16, "K": 128, "V": 128, "dtype": "bf16", "init": True},
        # a layer of 16 heads with 128-wide keys and values over a batch of prompts
        {"name": "prompt_layer_bf16", "op": "prompt", "lens": ",".join(["2048"] * 8), "H": 16,
         "G": 16, "K": 128, "V": 128, "dtype": "bf16", "init": False},
        # streaming prefill of one very long sequence, keys shared by all heads
        {"name": "prompt_long_bf16", "op": "prompt", "lens": "65536", "H": 32, "G": 1, "K": 128,
         "V": 64, "dtype": "bf16", "init": True},
        # a training step of a small fp32 model on packed ragged documents
        {"name": "train_ragged_fp32", "op": "train", "lens": "257,640,5,1,701", "H": 6, "G": 2,
         "K": 64, "V": 64, "dtype": "fp32", "init": True},
        # a training step of a small model's layer, grouped keys
        {"name": "train_grouped_bf16", "op": "train", "lens": "2048,2048,2048,2048", "H": 24,
         "G": 8, "K": 128, "V": 64, "dtype": "bf16", "init": False},
        # a training step of a large layer on packed documents
        {"name": "train_packed_bf16", "op": "train", "lens": "9000,5461,1923", "H": 32, "G": 32,
         "K": 128, "V": 128, "dtype": "bf16", "init": False},
        # one user's next token
        {"name": "step_one_bf16", "op": "step", "batch": 1, "H": 32, "G": 32, "K": 128, "V": 128,
         "dtype": "bf16"},
        # the next token of a full serving batch, grouped keys
        {"name": "step_batch_bf16", "op": "step", "batch": 200, "H": 32, "G": 8, "K": 128,
         "V": 64, "dtype": "bf16"},
        # the norm in front of a block for the tokens of three sequences
        {"name": "addnorm_tokens_bf16", "op": "addnorm", "rows": 3, "dim": 2560, "dtype": "bf16",
         "stream": "bf16", "scaled": False, "train": False},
        # a training step's norm with a scaled residual branch, the stream in fp32
        {"name": "addnorm_train_bf16", "op": "addnorm", "rows": 8191, "dim": 2560,
         "dtype": "bf16", "stream": "fp32", "scaled": True, "train": True},
        # the per-head norm and gate behind the mixer of a large layer's prompt
        {"name": "gatenorm_heads_bf16", "op": "gatenorm", "rows": 16384, "dim": 5120, "group": 64,
         "shared": True, "gate": "silu", "first": False, "dtype": "bf16", "side": "bf16",
         "train": False},
        # a training step's gate and norm over the whole inner width; the
        # mixer gives fp32
        {"name": "gatenorm_train_mixed", "op": "gatenorm", "rows": 8192, "dim": 1536,
         "group": 1536, "shared": False, "gate": "silu", "first": True, "dtype": "fp32",
         "side": "bf16", "train": True},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng):
    G = rng.choice([1, 2, 3, 4, 8, 16])
    return G * rng.choice([1, 1, 2, 3]), G


def draw(rng):
    op = rng.choice(["prompt", "train", "step", "addnorm", "gatenorm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("prompt", "train"):
        H, G = _heads(rng)
        total = _spread(rng, 1, 16384 if dtype == "bf16" else 4096)
        lens, left = [], total
        for _ in range(rng.choice([0, 0, 1, 3, 9])):
            n = rng.randint(0, left)
            lens.append(n)
            left -= n
        return {"op": op, "lens": ",".join(map(str, lens + [left])), "H": H, "G": G,
                "K": rng.choice([64, 128]), "V": rng.choice([64, 128]), "dtype": dtype,
                "init": rng.random() < 0.5}
    if op == "step":
        H, G = _heads(rng)
        return {"op": op, "batch": _spread(rng, 1, 200), "H": H, "G": G,
                "K": rng.choice([64, 128]), "V": rng.choice([64, 128]), "dtype": dtype}
    rows = _spread(rng, 1, 8192)
    train = rng.random() < 0.5
    if op == "addnorm":
        return {"op": op, "rows": rows, "dim": _spread(rng, 32, 5120), "dtype": dtype,
                "stream": rng.choice(["bf16", "fp32"]), "scaled": rng.random() < 0.5,
                "train": train}
    group = rng.choice([64, 128, _spread(rng, 32, 2560)])
    return {"op": op, "rows": rows, "dim": group * rng.choice([1, 2, 5, 20] if group <= 128 else [1, 2]),
            "group": group, "shared": rng.random() < 0.5, "gate": rng.choice(["silu", "sigmoid"]),
            "first": rng.random() < 0.5, "dtype": dtype, "side": rng.choice(["bf16", "fp32"]),
            "train": train}


# ----------------------------------------------------------------- inputs
def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    s = {"case": dict(case)}
    dt = TYPES[case["dtype"]]
    if case["op"] in ("prompt", "train", "step"):
        H, G, K, V = (case[n] for n in "HGKV")
        # slopes 2^(-8 (h+1) / H): the decays of a model with a span from one
        # token to some hundreds
        s["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H).float()
        s["scale"] = K ** -0.5
    if case["op"] == "step":
        b = case["batch"]
        s |= {"q": normal(b, G, K, dtype=dt), "k": normal(b, G, K, dtype=dt),
              "v": normal(b, H, V, dtype=dt), "state": normal(b, H, K, V, std=4.0),
              "o": torch.empty(b, H, V, dtype=dt, device=DEV)}
    elif case["op"] in ("prompt", "train"):
        lens = _lens(case)
        T, n = sum(lens), len(lens)
        s |= {"q": normal(1, T, G, K, dtype=dt), "k": normal(1, T, G, K, dtype=dt),
              "v": normal(1, T, H, V, dtype=dt), "longest": max(lens),
              "cu": torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32,
                                 device=DEV),
              "init": normal(n, H, K, V) if case["init"] else None}
        if case["op"] == "train":
            s |= {"do": normal(1, T, H, V, dtype=dt),
                  "dfinal": normal(n, H, K, V, std=0.1) if case["init"] else None}
    else:
        rows, D = case["rows"], case["dim"]
        s["x"] = normal(rows, D, dtype=dt)
        if case["op"] == "addnorm":
            st = TYPES[case["stream"]]
            s |= {"residual": normal(rows, D, dtype=st, std=3.0),
                  "scale": normal(D, std=0.1) + 0.5 if case["scaled"] else None,
                  "weight": normal(D, std=0.2) + 1.0}
            if case["train"]:
                s |= {"dy": normal(rows, D, dtype=dt), "dh": normal(rows, D, dtype=st)}
        else:
            sd = TYPES[case["side"]]
            s |= {"z": normal(rows, D, dtype=sd),
                  "weight": normal(case["group"] if case["shared"] else D, std=0.2) + 1.0}
            if case["train"]:
                s["dy"] = normal(rows, D, dtype=sd)
    return s


# ------------------------------------------------------------ plain forms
def _pad(x, cu, longest, heads):
    """Packed rows [1, T, n, D] as [nseq, heads, chunks, CHUNK, D] in 32 bits, zeros past each end."""
    n = max(1, -(-longest // CHUNK)) * CHUNK
    at = torch.arange(n, device=x.device)
    start, length = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    rows = (start[:, None] + at).clamp(max=x.shape[1] - 1)
    x = torch.where((at < length[:, None])[..., None, None], x[0].float()[rows], 0.0)
    x = x.repeat_interleave(heads // x.shape[2], dim=2).transpose(1, 2)
    return x.reshape(x.shape[0], heads, n // CHUNK, CHUNK, -1)


def _unpad(x, cu, T, dtype):
    """The packed rows [1, T, n, D] of a padded [nseq, n, chunks, CHUNK, D], rounded."""
    x = x.flatten(2, 3).transpose(1, 2)
    at = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu[1:].long(), at, right=True)
    return x[seq, at - cu.long()[seq]].to(dtype)[None]


def _powers(log_decay, exponents):
    """exp(log_decay * exponents) for each head, 0 for negative exponents; angles in 64 bits."""
    e = log_decay.double().view(-1, *[1] * exponents.dim()) * exponents.double()
    return torch.where(exponents >= 0, torch.exp(e), 0.0).float()


class _Decays:
    """The decay factors that the chunked forms share."""

    def __init__(self, s, chunks):
        ld, dev = s["log_decay"], s["log_decay"].device
        i = torch.arange(CHUNK, device=dev)
        c = torch.arange(chunks, device=dev)
        t = torch.arange(chunks * CHUNK, device=dev)
        length = (s["cu"][1:] - s["cu"][:-1]).long()
        self.inside = _powers(ld, i[:, None] - i)[:, None]              # [H, 1, C, C]
        self.after = _powers(ld, i + 1)[:, None, :, None]               # [H, 1, C, 1]
        self.before = _powers(ld, CHUNK - 1 - i)[:, None, :, None]
        self.chunks = _powers(ld, CHUNK * (c[:, None] - 1 - c))         # [H, nc, nc], c' < c
        self.start = _powers(ld, CHUNK * c)[:, :, None, None]           # [H, nc, 1, 1]
        self.to_end = _powers(ld, length[:, None] - 1 - t).transpose(0, 1)[..., None]
        self.from_start = _powers(ld, t + 1)[:, :, None]                # [H, L, 1]
        self.whole = _powers(ld, length).t()[..., None, None]           # [nseq, H, 1, 1]


def _chunk_states(k, v, d, init):
    """Each chunk's starting state [nseq, H, nc, K, V]."""
    each = (k * d.before).transpose(-1, -2) @ v
    states = (d.chunks @ each.flatten(-2)).view_as(each)
    return states if init is None else states + d.start * init[:, :, None]


def _plain_prompt(s):
    H, T = s["v"].shape[2], s["v"].shape[1]
    q, k, v = (_pad(s[n], s["cu"], s["longest"], H) for n in "qkv")
    d = _Decays(s, q.shape[2])
    o = ((q @ k.transpose(-1, -2)) * d.inside) @ v
    o = o + (q * d.after) @ _chunk_states(k, v, d, s["init"])
    final = (k.flatten(2, 3) * d.to_end).transpose(-1, -2) @ v.flatten(2, 3)
    if s["init"] is not None:
        final = final + d.whole * s["init"]
    return _unpad(o * s["scale"], s["cu"], T, s["v"].dtype), final


def _plain_gradients(s):
    H, T, G = s["v"].shape[2], s["v"].shape[1], s["q"].shape[2]
    q, k, v, do = (_pad(s[n], s["cu"], s["longest"], H) for n in ("q", "k", "v", "do"))
    d = _Decays(s, q.shape[2])
    do_s = do * s["scale"]
    scores, back = (q @ k.transpose(-1, -2)) * d.inside, (do_s @ v.transpose(-1, -2)) * d.inside
    states = _chunk_states(k, v, d, s["init"])
    dq = back @ k + (do_s * d.after) @ states.transpose(-1, -2)
    each = (q * d.after).transpose(-1, -2) @ do_s
    later = (d.chunks.transpose(-1, -2) @ each.flatten(-2)).view_as(each)
    dk = back.transpose(-1, -2) @ q + (v * d.before) @ later.transpose(-1, -2)
    dv = scores.transpose(-1, -2) @ do_s + (k * d.before) @ later
    dinit = (q.flatten(2, 3) * d.from_start).transpose(-1, -2) @ do_s.flatten(2, 3)
    if s["dfinal"] is not None:
        end = d.to_end.view(*d.to_end.shape[:2], -1, CHUNK, 1)
        dk = dk + (v * end) @ s["dfinal"][:, :, None].transpose(-1, -2)
        dv = dv + (k * end) @ s["dfinal"][:, :, None]
        dinit = dinit + d.whole * s["dfinal"]
    dq, dk = (x.unflatten(1, (G, H // G)).sum(2) for x in (dq, dk))
    dq, dk, dv = (_unpad(x, s["cu"], T, s["v"].dtype) for x in (dq, dk, dv))
    return dq, dk, dv, dinit


def _plain_step(s):
    H = s["v"].shape[1]
    q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], dim=1) for n in "qk")
    lam = torch.exp(s["log_decay"].double()).float()
    s["state"].copy_(s["state"] * lam[:, None, None] + k[..., None] * s["v"].float()[:, :, None])
    s["o"].copy_(((q[..., None] * s["state"]).sum(2) * s["scale"]))
    return s["o"], s["state"]


def _plain_addnorm(s):
    x, h = s["x"].float(), s["residual"].float()
    h = h + (x if s["scale"] is None else x * s["scale"])
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * rstd
    out = [(n * s["weight"]).to(s["x"].dtype), h.to(s["residual"].dtype)]
    if "dy" in s:
        dy = s["dy"].float()
        u = dy * s["weight"]
        g = s["dh"].float() + rstd * (u - n * (u * n).mean(-1, keepdim=True))
        dx = g if s["scale"] is None else g * s["scale"]
        out += [dx.to(s["x"].dtype), g.to(s["residual"].dtype), (dy * n).sum(0)]
        if s["scale"] is not None:
            out.append((g * x).sum(0))
    return out


def _plain_gatenorm(s):
    c = s["case"]
    rows, D, group = c["rows"], c["dim"], c["group"]
    x, z = (s[n].float().view(rows, D // group, group) for n in "xz")
    w = s["weight"].view(-1, group)
    sig = torch.sigmoid(z)
    act = z * sig if c["gate"] == "silu" else sig
    u = x * act if c["first"] else x
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    n = u * rstd
    y = n * w if c["first"] else n * w * act
    out = [y.view(rows, D).to(s["z"].dtype)]
    if "dy" in s:
        dy = s["dy"].float().view_as(x)
        dn = dy if c["first"] else dy * act
        wdn = dn * w
        du = rstd * (wdn - n * (wdn * n).mean(-1, keepdim=True))
        dx, dact = (du * act, du * x) if c["first"] else (du, dy * n * w)
        dsig = sig * (1 - sig)
        dz = dact * (sig + z * dsig if c["gate"] == "silu" else dsig)
        dw = (dn * n).sum(0)
        dw = dw.sum(0) if c["shared"] else dw.reshape(-1)
        out += [dx.reshape(rows, D).to(s["x"].dtype), dz.reshape(rows, D).to(s["z"].dtype), dw]
    return out


# -------------------------------------------------------------------- run
def _own(s):
    import mamba_ssd_chunked_fwd_amd as ssd
    c = s["case"]
    if c["op"] in ("prompt", "train"):
        out = list(ssd.linattn(s["q"], s["k"], s["v"], s["log_decay"], s["init"], s["cu"],
                               s["scale"]))
        if c["op"] == "train":
            out += ssd.linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"],
                                        s["dfinal"], s["init"], s["cu"], s["scale"])
        return out
    if c["op"] == "step":
        ssd.ssd_linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["o"],
                             s["scale"])
        return s["o"], s["state"]
    if c["op"] == "addnorm":
        out = list(ssd.add_norm(s["x"], s["residual"], s["scale"], s["weight"], EPS))
        if c["train"]:
            dx, dresidual, dscale, dweight = ssd.add_norm_backward(
                s["x"], s["residual"], s["scale"], s["weight"], s["dy"], s["dh"], EPS)
            out += [dx, dresidual, dweight] + ([] if dscale is None else [dscale])
        return out
    out = [ssd.gated_norm(s["x"], s["z"], s["weight"], EPS, c["group"], c["gate"], c["first"])]
    if c["train"]:
        out += ssd.gated_norm_backward(s["x"], s["z"], s["weight"], s["dy"], EPS, c["group"],
                                       c["gate"], c["first"])
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "prompt":
        return list(_plain_prompt(state))
    if op == "train":
        return [*_plain_prompt(state), *_plain_gradients(state)]
    return {"step": _plain_step, "addnorm": _plain_addnorm, "gatenorm": _plain_gatenorm}[op](state)


def work(case):
    e = {"bf16": 2, "fp32": 4}
    op = case["op"]
    if op in ("prompt", "train", "step"):
        H, G, K, V = (case[n] for n in "HGKV")
        n = case["batch"] if op == "step" else len(_lens(case))
        T = n if op == "step" else sum(_lens(case))
        el, state = e[case["dtype"]], 4 * n * H * K * V
        qk, v = el * T * G * K, el * T * H * V
        # the recurrence: a rank-one update and a product with the state for
        # each token (as many again, and half, for the three gradients)
        nbytes, flops = 2 * qk + 2 * v, 4.0 * T * H * K * V
        nbytes += state * (2 if op == "step" or case["init"] else 1)
        if op == "train":
            nbytes += 4 * qk + 3 * v + state * (3 if case["init"] else 1)
            flops += 10.0 * T * H * K * V
        return {"bytes": nbytes, "flops": flops}
    n, D = case["rows"] * case["dim"], case["dim"]
    a = e[case["dtype"]]
    if op == "addnorm":
        b = e[case["stream"]]
        nbytes = n * (2 * a + 2 * b) + 4 * D
        if case["train"]:
            nbytes += n * (3 * a + 3 * b) + 12 * D
        return {"bytes": nbytes, "flops": n * (22 if case["train"] else 6)}
    b = e[case["side"]]
    nbytes = n * (a + 2 * b) + 4 * D
    if case["train"]:
        nbytes += n * (2 * a + 3 * b) + 8 * D
    return {"bytes": nbytes, "flops": n * (30 if case["train"] else 9)}


# ------------------------------------------------------------------ exact
def _exact_linattn(s, train):
    """The recurrence token by token, and its adjoint from the last token to the first."""
    cu = s["cu"].tolist()
    n, H, G = len(cu) - 1, s["v"].shape[2], s["q"].shape[2]
    K, V, T = s["q"].shape[3], s["v"].shape[3], s["v"].shape[1]
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    group = torch.arange(H, device=DEV) // (H // G)
    lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device=DEV)
    first = torch.tensor(cu[:-1], device=DEV)
    S = torch.zeros(n, H, K, V, dtype=torch.float64, device=DEV)
    if s["init"] is not None:
        S += s["init"]
    q, k, v = s["q"][0], s["k"][0], s["v"][0]
    o = torch.zeros(T, H, V, dtype=torch.float64, device=DEV)
    if train:
        do = s["do"][0]
        dq, dk = (torch.zeros(T, G, K, dtype=torch.float64, device=DEV) for _ in range(2))
        dv = torch.zeros_like(o)
    order = torch.argsort(lens, descending=True)   # the sequences still running lead
    first, S = first[order], S[order]
    running = [int((lens > t).sum()) for t in range(s["longest"])]
    for t, m in enumerate(running):
        at = first[:m] + t
        S[:m].mul_(lam).add_(k[at][:, group].double()[..., None] * v[at].double()[:, :, None])
        o[at] = s["scale"] * (q[at][:, group].double()[:, :, None] @ S[:m])[:, :, 0]
        if train:
            back = (S[:m] @ do[at].double()[..., None])[..., 0] * s["scale"]
            dq[at] = back.view(m, G, -1, K).sum(2)
    back_order = torch.argsort(order)
    out = [o[None], S[back_order]]
    if train:
        R = torch.zeros_like(S)
        if s["dfinal"] is not None:
            R += s["dfinal"][order]
        # R holds lam * dS_{t+1}: dfinal itself past the last token
        for t in range(s["longest"] - 1, -1, -1):
            m = running[t]
            at = first[:m] + t
            R[:m].add_(s["scale"] * q[at][:, group].double()[..., None] * do[at].double()[:, :, None])
            dk[at] = (R[:m] @ v[at].double()[..., None])[..., 0].view(m, G, -1, K).sum(2)
            dv[at] = (k[at][:, group].double()[:, :, None] @ R[:m])[:, :, 0]
            R[:m].mul_(lam)
        out += [dq[None], dk[None], dv[None], R[back_order]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "train"):
        lens = _lens(case)
        passes = 3 if op == "train" else 1
        cells = case["H"] * case["K"] * case["V"]
        if passes * (max(lens) * 100e-6 + sum(lens) * cells * 8 * 8 / 2e12) > 18:
            return None
        return _exact_linattn(s, op == "train")
    if op == "step":
        H = case["H"]
        q, k = (s[n].double().repeat_interleave(H // case["G"], dim=1) for n in "qk")
        S = s["state"].double() * torch.exp(s["log_decay"].double())[:, None, None]
        S = S + k[..., None] * s["v"].double()[:, :, None]
        return [(q[:, :, None] @ S)[:, :, 0] * s["scale"], S]
    leaf = {n: s[n].double().requires_grad_() for n in ("x", "residual", "scale", "weight", "z")
            if s.get(n) is not None}
    if op == "addnorm":
        h = leaf["residual"] + leaf["x"] * leaf.get("scale", 1.0)
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * leaf["weight"]
        out = [y.detach(), h.detach()]
        if case["train"]:
            want = [leaf["x"], leaf["residual"], leaf["weight"]]
            want += [leaf["scale"]] if case["scaled"] else []
            out += torch.autograd.grad([y, h], want, [s["dy"].double(), s["dh"].double()])
        return out
    shape = (case["rows"], case["dim"] // case["group"], case["group"])
    x, z = leaf["x"].view(shape), leaf["z"].view(shape)
    act = z / (1 + torch.exp(-z)) if case["gate"] == "silu" else 1 / (1 + torch.exp(-z))
    u = x * act if case["first"] else x
    y = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * leaf["weight"].view(-1, shape[2])
    y = (y if case["first"] else y * act).reshape(case["rows"], case["dim"])
    out = [y.detach()]
    if case["train"]:
        out += torch.autograd.grad(y, [leaf["x"], leaf["z"], leaf["weight"]], s["dy"].double())
    return out
