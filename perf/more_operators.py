"""The operators of a recurrent block with a selective state space, as cases to be measured.

  conv      the short causal convolution over whole (packed) sequences
  convstep  its single-token form, the last inputs kept in a state
  scan      the selective scan over whole (packed) sequences
  scanstep  its recurrent form: one token for every sequence of a batch
  normq     residual add and norm, the output in 8 bits with scales

Where ``own`` is false, ``run`` computes them in elementary torch operations
in 32 bits; where it is true it calls the package.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few short requests prefilled together from cached states, one of
        # them a single token and one empty: latency counts
        {"name": "conv_ragged_bf16", "op": "conv", "lens": "1,37,64,130,0,411", "dim": 1536,
         "width": 4, "silu": True, "bias": True, "dtype": "bf16", "init": True, "train": False},
        # a training step of a large layer: x, B and C filtered together
        {"name": "conv_train_bf16", "op": "conv", "lens": "9000,5461,1923", "dim": 5376,
         "width": 4, "silu": True, "bias": True, "dtype": "bf16", "init": False, "train": True},
        # one user's next token
        {"name": "convstep_one_bf16", "op": "convstep", "batch": 1, "dim": 2560, "width": 4,
         "silu": True, "bias": True, "dtype": "bf16"},
        # the next token of a full serving batch
        {"name": "convstep_batch_bf16", "op": "convstep", "batch": 200, "dim": 5376, "width": 4,
         "silu": True, "bias": True, "dtype": "bf16"},
        # the short requests' scan
        {"name": "scan_ragged_bf16", "op": "scan", "lens": "1,37,64,130,0,411", "dim": 1536,
         "N": 16, "G": 1, "skip": True, "gate": True, "bias": True, "dtype": "bf16",
         "init": True, "train": False},
        # streaming prefill of one long sequence by a large layer
        {"name": "scan_long_bf16", "op": "scan", "lens": "32768", "dim": 5120, "N": 16, "G": 1,
         "skip": True, "gate": True, "bias": True, "dtype": "bf16", "init": True, "train": False},
        # a training step of a small fp32 model on packed ragged documents
        {"name": "scan_train_ragged_fp32", "op": "scan", "lens": "257,640,5,1,701", "dim": 768,
         "N": 16, "G": 1, "skip": True, "gate": True, "bias": True, "dtype": "fp32",
         "init": True, "train": True},
        # a training step of a layer on packed documents
        {"name": "scan_train_packed_bf16", "op": "scan", "lens": "9000,5461,1923", "dim": 2560,
         "N": 16, "G": 1, "skip": True, "gate": True, "bias": True, "dtype": "bf16",
         "init": False, "train": True},
        # one user's next token
        {"name": "scanstep_one_bf16", "op": "scanstep", "batch": 1, "dim": 2560, "N": 16, "G": 1,
         "skip": True, "gate": True, "bias": True, "dtype": "bf16"},
        # the next token of a full serving batch
        {"name": "scanstep_batch_bf16", "op": "scanstep", "batch": 200, "dim": 5120, "N": 16,
         "G": 1, "skip": True, "gate": True, "bias": True, "dtype": "bf16"},
        # the norm in front of a block whose projection takes 8 bits, for the
        # tokens of three sequences, a scale for each row
        {"name": "normq_tokens_e4m3", "op": "normq", "rows": 3, "dim": 2560, "group": 2560,
         "code": "e4m3", "dtype": "bf16", "stream": "bf16", "scaled": False},
        # the same for a prompt, a scale for each 128 channels, the stream in fp32
        {"name": "normq_prompt_e4m3", "op": "normq", "rows": 16384, "dim": 5120, "group": 128,
         "code": "e4m3", "dtype": "bf16", "stream": "fp32", "scaled": True},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _split(rng, total):
    """Lengths of some sequences, empty ones among them, of `total` tokens in all."""
    lens, left = [], total
    for _ in range(rng.choice([0, 0, 1, 3, 9])):
        n = rng.randint(0, left)
        lens.append(n)
        left -= n
    return ",".join(map(str, lens + [left]))


def draw(rng):
    op = rng.choice(["conv", "conv", "convstep", "scan", "scan", "scan", "scanstep", "normq"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    some = {"silu": rng.random() < 0.8, "bias": rng.random() < 0.8}
    if op in ("conv", "convstep"):
        c = {"op": op, "dim": _spread(rng, 32, 5376), "width": rng.choice([2, 3, 4, 4]),
             "dtype": dtype, **some}
        if op == "convstep":
            return c | {"batch": _spread(rng, 1, 200)}
        return c | {"lens": _split(rng, _spread(rng, 1, 8192)), "init": rng.random() < 0.5,
                    "train": rng.random() < 0.5}
    if op in ("scan", "scanstep"):
        G = rng.choice([1, 1, 1, 2, 4])
        N = rng.choice([16, 16, 16, 8, 32, 64])
        c = {"op": op, "dim": G * _spread(rng, 32, 2560 // G), "N": N, "G": G,
             "skip": rng.random() < 0.8, "gate": rng.random() < 0.8, "bias": some["bias"],
             "dtype": dtype}
        if op == "scanstep":
            return c | {"batch": _spread(rng, 1, 200)}
        return c | {"lens": _split(rng, _spread(rng, 1, 16384 * 16 // max(N, 16) // 2)),
                    "init": rng.random() < 0.5, "train": rng.random() < 0.5}
    group = rng.choice([32, 64, 128, 0])
    dim = _spread(rng, 32, 5120)
    dim = dim if group == 0 else max(1, dim // group) * group
    return {"op": op, "rows": _spread(rng, 1, 8192), "dim": dim, "group": group or dim,
            "code": rng.choice(["e4m3", "e4m3", "int8"]), "dtype": dtype,
            "stream": rng.choice(["bf16", "fp32"]), "scaled": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs
def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    s = {"case": dict(case)}
    dt, D = TYPES[case["dtype"]], case["dim"]
    if "lens" in case:
        lens = _lens(case)
        T, n = sum(lens), len(lens)
        s |= {"longest": max(lens),
              "cu": torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32,
                                 device=DEV)}
        lead = (1, T)
    elif "batch" in case:
        n = case["batch"]
        lead = (n,)
    if case["op"] in ("conv", "convstep"):
        W = case["width"]
        # one projection gives x and the gate: x is its first half
        s |= {"x": normal(*lead, 2 * D, dtype=dt)[..., :D],
              "weight": normal(D, W, std=W ** -0.5),
              "bias": normal(D, std=0.1) if case["bias"] else None}
        if case["op"] == "convstep":
            s |= {"state": normal(n, W - 1, D, dtype=dt),
                  "y": torch.empty(n, D, dtype=dt, device=DEV)}
        else:
            s["init"] = normal(n, W - 1, D, dtype=dt) if case["init"] else None
            if case["train"]:
                s |= {"dy": normal(*lead, D, dtype=dt),
                      "dfinal": normal(n, W - 1, D, dtype=dt) if case["init"] else None}
    elif case["op"] in ("scan", "scanstep"):
        N, G = case["N"], case["G"]
        R = -(-D // 16) // 8 * 8 + 8          # the low-rank part in front of B and C
        proj = normal(*lead, R + 2 * G * N, dtype=dt)
        # time steps of 0.001 to 0.1 before the input's own part, decays of 1
        # to N for each
        step = torch.exp(torch.rand(D, generator=gen, device=DEV) * math.log(100.0)) * 1e-3
        s |= {"x": normal(*lead, D, dtype=dt), "dt": normal(*lead, D, dtype=dt, std=0.7),
              "A": -torch.arange(1, N + 1, device=DEV).float() * (1 + 0.1 * normal(D, N)).abs(),
              "B": proj[..., R:R + G * N].unflatten(-1, (G, N)),
              "C": proj[..., R + G * N:].unflatten(-1, (G, N)),
              "D": 1 + normal(D, std=0.2) if case["skip"] else None,
              "z": normal(*lead, 2 * D, dtype=dt)[..., D:] if case["gate"] else None,
              "dt_bias": torch.log(torch.expm1(step)) if case["bias"] else None}
        if not case["bias"]:
            s["dt"] = (s["dt"].float() - 4.0).to(dt)
        if case["op"] == "scanstep":
            s |= {"state": normal(n, D, N), "y": torch.empty(n, D, dtype=dt, device=DEV)}
        else:
            s["init"] = normal(n, D, N) if case["init"] else None
            if case["train"]:
                s |= {"dy": normal(*lead, D, dtype=dt),
                      "dfinal": normal(n, D, N, std=0.1) if case["init"] else None}
    else:
        rows = case["rows"]
        s |= {"x": normal(rows, D, dtype=dt),
              "residual": normal(rows, D, dtype=TYPES[case["stream"]], std=3.0),
              "scale": normal(D, std=0.1) + 0.5 if case["scaled"] else None,
              "weight": normal(D, std=0.2) + 1.0}
    return s


# ------------------------------------------------------------ plain forms
def _places(s, T):
    """The sequence of each packed row and its place in it."""
    at = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    return seq, at - s["cu"].long()[seq]


def _plain_conv(s):
    c = s["case"]
    W, D = c["width"], c["dim"]
    x, n, T = s["x"][0].float(), len(s["cu"]) - 1, s["x"].shape[1]
    before = torch.zeros(n, W - 1, D, device=DEV) if s["init"] is None else s["init"].float()
    # every sequence with its last inputs in front of it, one behind the other
    seq, place = _places(s, T)
    own_row = s["cu"][:-1].long()[seq] + (seq + 1) * (W - 1) + place
    front = s["cu"][:-1].long()[:, None] + torch.arange(n, device=DEV)[:, None] * (W - 1) \
        + torch.arange(W - 1, device=DEV)
    ext = torch.empty(T + n * (W - 1), D, device=DEV)
    ext[own_row], ext[front] = x, before
    bias = 0.0 if s["bias"] is None else s["bias"]
    pre = sum(ext[own_row - (W - 1) + k] * s["weight"][:, k] for k in range(W)) + bias
    sig = torch.sigmoid(pre)
    dt = s["x"].dtype
    y = pre * sig if c["silu"] else pre
    last = front + (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    out = [y.to(dt)[None], ext[last].to(dt)]
    if c["train"]:
        g = s["dy"][0].float()
        if c["silu"]:
            g = g * sig * (1 + pre * (1 - sig))
        dext = torch.zeros_like(ext)
        for k in range(W):
            dext[own_row - (W - 1) + k] += g * s["weight"][:, k]
        if s["dfinal"] is not None:
            dext.index_put_((last,), s["dfinal"].float(), accumulate=True)
        out += [dext[own_row].to(dt)[None],
                torch.stack([(g * ext[own_row - (W - 1) + k]).sum(0) for k in range(W)], 1)]
        if s["bias"] is not None:
            out.append(g.sum(0))
        if s["init"] is not None:
            out.append(dext[front].to(dt))
    return out


def _plain_convstep(s):
    ext = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    pre = (ext * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    s["y"].copy_(pre * torch.sigmoid(pre) if s["case"]["silu"] else pre)
    s["state"].copy_(ext[:, 1:])
    return s["y"], s["state"]


class _Chunks:
    """The inputs of a scan cut into chunks of `size` tokens, [sequences * chunks, size, ...];
    places past a sequence's end have a time step of 0."""

    def __init__(self, s):
        c = s["case"]
        T, n = s["x"].shape[1], len(s["cu"]) - 1
        self.seq, self.place = _places(s, T)
        self.size = max(1, math.isqrt(max(1, s["longest"])))
        self.number = max(1, -(-s["longest"] // self.size))
        self.n, self.T = n, T
        raw = s["dt"][0].float()
        if s["dt_bias"] is not None:
            raw = raw + s["dt_bias"]
        self.raw = raw
        # ln(1 + exp(raw)), formed in 64 bits where the exponential is small
        self.delta = torch.log1p(torch.exp(-raw.abs().double())).float() + raw.clamp(min=0)
        self.step = self.cut(self.delta)
        self.x = self.cut(s["x"][0].float())
        reps = c["dim"] // c["G"]
        self.B, self.C = (self.cut(s[k][0].float().flatten(1)).unflatten(-1, (c["G"], c["N"]))
                          for k in "BC")
        self.heads = lambda t: t.repeat_interleave(reps, dim=-2)
        self.A = s["A"]

    def cut(self, t):
        out = torch.zeros(self.n, self.number * self.size, *t.shape[1:], device=DEV)
        out[self.seq, self.place] = t
        return out.view(self.n * self.number, self.size, *t.shape[1:])

    def rows(self, t):
        t = t.reshape(self.n, self.number * self.size, *t.shape[2:])
        return t[self.seq, self.place]

    def decay(self, i):
        return torch.exp(self.step[:, i, :, None] * self.A)

    def add(self, i):
        return (self.step[:, i] * self.x[:, i])[..., None] * self.heads(self.B[:, i])

    def whole(self):
        """Each chunk's decay, the sum of its time steps in 64 bits."""
        total = self.step.double().sum(1)
        return torch.exp(total[..., None] * self.A.double()).float()


def _plain_scan(s):
    c = s["case"]
    ch = _Chunks(s)
    D, N = c["dim"], c["N"]
    local = torch.zeros(ch.n * ch.number, D, N, device=DEV)
    for i in range(ch.size):
        local = local * ch.decay(i) + ch.add(i)
    whole = ch.whole().view(ch.n, ch.number, D, N)
    local = local.view(ch.n, ch.number, D, N)
    h = torch.zeros(ch.n, D, N, device=DEV) if s["init"] is None else s["init"]
    starts = torch.empty_like(local)
    for k in range(ch.number):
        starts[:, k] = h
        h = h * whole[:, k] + local[:, k]
    final, h = h, starts.view(-1, D, N)
    keep, y = [h], torch.empty_like(ch.x)
    for i in range(ch.size):
        h = h * ch.decay(i) + ch.add(i)
        y[:, i] = (h * ch.heads(ch.C[:, i])).sum(-1)
        if c["train"]:
            keep.append(h)
    x = s["x"][0].float()
    u = ch.rows(y)
    if s["D"] is not None:
        u = u + x * s["D"]
    out, dt = u, s["x"].dtype
    if s["z"] is not None:
        z = s["z"][0].float()
        sig = torch.sigmoid(z)
        out = u * z * sig
    result = [out.to(dt)[None], final]
    if not c["train"]:
        return result

    # gradients
    du = s["dy"][0].float()
    dz = None
    if s["z"] is not None:
        dz = du * u * sig * (1 + z * (1 - sig))
        du = du * z * sig
    g = ch.cut(du)
    local = torch.zeros(ch.n * ch.number, D, N, device=DEV)
    for i in reversed(range(ch.size)):
        local = (local + ch.heads(ch.C[:, i]) * g[:, i, :, None]) * ch.decay(i)
    local = local.view(ch.n, ch.number, D, N)
    r = torch.zeros(ch.n, D, N, device=DEV) if s["dfinal"] is None else s["dfinal"]
    ends = torch.empty_like(local)
    for k in reversed(range(ch.number)):
        ends[:, k] = r
        r = r * whole[:, k] + local[:, k]
    dinit, r = r, ends.view(-1, D, N)
    dB, dC = torch.empty_like(ch.B), torch.empty_like(ch.C)
    dxs, dstep = torch.empty_like(ch.x), torch.empty_like(ch.x)
    dA = torch.zeros(ch.n * ch.number, D, N, device=DEV)

    def groups(t):
        return t.unflatten(1, (c["G"], D // c["G"])).sum(2)

    for i in reversed(range(ch.size)):
        decay, step, xi = ch.decay(i), ch.step[:, i], ch.x[:, i]
        dh = r + ch.heads(ch.C[:, i]) * g[:, i, :, None]
        dC[:, i] = groups(g[:, i, :, None] * keep[i + 1])
        dB[:, i] = groups(dh * (step * xi)[..., None])
        part = (dh * ch.heads(ch.B[:, i])).sum(-1)
        gone = dh * keep[i] * decay
        dxs[:, i] = part * step
        dstep[:, i] = part * xi + (gone * ch.A).sum(-1)
        dA += gone * step[..., None]
        r = dh * decay
    dx = ch.rows(dxs)
    if s["D"] is not None:
        dx = dx + du * s["D"]
    ddt = ch.rows(dstep) * torch.sigmoid(ch.raw)
    result += [dx.to(dt)[None], ddt.to(dt)[None], dA.sum(0), ch.rows(dB).to(dt)[None],
               ch.rows(dC).to(dt)[None]]
    if s["D"] is not None:
        result.append((du * x).sum(0))
    if dz is not None:
        result.append(dz.to(dt)[None])
    if s["dt_bias"] is not None:
        result.append(ddt.sum(0))
    if s["init"] is not None:
        result.append(dinit)
    return result


def _plain_scanstep(s):
    c = s["case"]
    raw = s["dt"].float() if s["dt_bias"] is None else s["dt"].float() + s["dt_bias"]
    step = torch.log1p(torch.exp(-raw.abs().double())).float() + raw.clamp(min=0)
    B, C = (s[k].float().repeat_interleave(c["dim"] // c["G"], dim=1) for k in "BC")
    x = s["x"].float()
    s["state"].copy_(s["state"] * torch.exp(step[..., None] * s["A"]) + (step * x)[..., None] * B)
    u = (s["state"] * C).sum(-1)
    if s["D"] is not None:
        u = u + x * s["D"]
    if s["z"] is not None:
        z = s["z"].float()
        u = u * z * torch.sigmoid(z)
    s["y"].copy_(u)
    return s["y"], s["state"]


def _values(codes, scales, group):
    """The values that codes of 8 bits and their scales stand for."""
    return (codes.float().unflatten(-1, (-1, group)) * scales[..., None]).flatten(-2)


def _plain_normq(s):
    # in 64 bits: a value next to the border of two codes takes the nearer one
    c = s["case"]
    kind, top = CODES[c["code"]]
    x, h = s["x"].double(), s["residual"].double()
    h = h + (x if s["scale"] is None else x * s["scale"])
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    y = y.unflatten(-1, (-1, c["group"]))
    amax = y.abs().amax(-1)
    codes = y * torch.where(amax > 0, top / amax, 0.0)[..., None]
    if c["code"] == "e4m3":        # to 4 significant bits at once, not to 32 bits first
        part, power = torch.frexp(codes)
        power = power.clamp(min=-5) - 4
        part = torch.ldexp(codes, -power)
        codes = torch.ldexp(torch.round(part), power)
    codes = torch.round(codes) if c["code"] == "int8" else codes
    codes = codes.to(kind).flatten(-2)
    scales = (amax / top).float()
    return [_values(codes, scales, c["group"]), scales, h.to(s["residual"].dtype)]


# -------------------------------------------------------------------- run
def _own(s):
    import mamba_ssd_chunked_fwd_amd as ssd
    c = s["case"]
    if c["op"] == "conv":
        act = "silu" if c["silu"] else None
        out = list(ssd.short_conv(s["x"], s["weight"], s["bias"], s["init"], s["cu"], act))
        if c["train"]:
            out += ssd.short_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], s["dfinal"],
                                           s["init"], s["cu"], act)
    elif c["op"] == "convstep":
        ssd.ssd_short_conv_step(s["x"], s["weight"], s["bias"], s["state"], s["y"],
                                "silu" if c["silu"] else None)
        out = [s["y"], s["state"]]
    elif c["op"] == "scan":
        a = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"])
        out = list(ssd.selective_scan(*a, s["init"], s["cu"]))
        if c["train"]:
            out += ssd.selective_scan_backward(*a, s["dy"], s["dfinal"], s["init"], s["cu"])
    elif c["op"] == "scanstep":
        ssd.ssd_selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                    s["dt_bias"], s["state"], s["y"])
        out = [s["y"], s["state"]]
    else:
        codes, scales, h = ssd.add_norm_quant(s["x"], s["residual"], s["scale"], s["weight"], EPS,
                                              CODES[c["code"]][0], c["group"])
        out = [_values(codes, scales, c["group"]), scales, h]
    return [t for t in out if t is not None]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return list({"conv": _plain_conv, "convstep": _plain_convstep, "scan": _plain_scan,
                 "scanstep": _plain_scanstep, "normq": _plain_normq}[op](state))


def work(case):
    e = {"bf16": 2, "fp32": 4}
    op, D, el = case["op"], case["dim"], e[case["dtype"]]
    n = case.get("batch", 0) or len(case.get("lens", "").split(","))
    T = sum(_lens(case)) if "lens" in case else n
    if op in ("conv", "convstep"):
        W = case["width"]
        state = el * n * (W - 1) * D
        weights = 4 * D * (W + (1 if case["bias"] else 0))
        if op == "convstep":
            return {"bytes": 2 * el * n * D + 2 * state + weights, "flops": n * D * (2 * W + 5)}
        nbytes = 2 * el * T * D + state * (2 if case["init"] else 1) + weights
        flops = T * D * (2 * W + 5)
        if case["train"]:
            nbytes += 3 * el * T * D + weights * 2 + state * (3 if case["init"] else 0)
            flops += T * D * (6 * W + 12)
        return {"bytes": nbytes, "flops": flops}
    if op in ("scan", "scanstep"):
        N, G = case["N"], case["G"]
        z = 1 if case["gate"] else 0
        state, bc = 4 * n * D * N, 2 * el * T * G * N
        weights = 4 * D * (N + 2)
        nbytes = el * T * D * (3 + z) + bc + weights
        nbytes += state * (2 if op == "scanstep" or case["init"] else 1)
        # a product for the exponent, the exponential, the new state and the output
        flops = T * D * (7.0 * N + 12)
        if op == "scan" and case["train"]:
            nbytes += el * T * D * (5 + 2 * z) + 2 * bc + 2 * weights
            nbytes += state * (3 if case["init"] else 0)
            flops += T * D * (18.0 * N + 30)
        return {"bytes": nbytes, "flops": flops}
    rows = case["rows"]
    nbytes = rows * (D * (el + 2 * e[case["stream"]] + 1) + 4 * (D // case["group"]))
    return {"bytes": nbytes + 8 * D, "flops": rows * D * 9}


# ------------------------------------------------------------------ exact
def _exact_conv(s):
    c = s["case"]
    W, cu = c["width"], s["cu"].tolist()
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "weight", "bias", "init")
            if s[k] is not None}
    ys, finals = [], []
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        front = leaf["init"][i] if "init" in leaf \
            else torch.zeros(W - 1, c["dim"], dtype=torch.float64, device=DEV)
        rows = torch.cat([front, leaf["x"][0, a:b]])
        y = torch.zeros(b - a, c["dim"], dtype=torch.float64, device=DEV)
        for k in range(W):
            y = y + leaf["weight"][:, k] * rows[k:k + b - a]
        y = y + leaf["bias"] if "bias" in leaf else y
        ys.append(y / (1 + torch.exp(-y)) if c["silu"] else y)
        finals.append(rows[b - a:])
    y, final = torch.cat(ys)[None], torch.stack(finals)
    out = [y.detach(), final.detach()]
    if c["train"]:
        ends, seeds = [y], [s["dy"].double()]
        if s["dfinal"] is not None:
            ends, seeds = ends + [final], seeds + [s["dfinal"].double()]
        out += torch.autograd.grad(ends, list(leaf.values()), seeds)
    return out


def _exact_scan(s):
    """The recurrence token by token, and its adjoint from the last token to the first."""
    c = s["case"]
    cu = s["cu"].tolist()
    D, N, G, T, n = c["dim"], c["N"], c["G"], s["x"].shape[1], len(cu) - 1
    lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device=DEV)
    order = torch.argsort(lens, descending=True)   # the sequences still running lead
    first = torch.tensor(cu[:-1], device=DEV)[order]
    running = [int((lens > t).sum()) for t in range(s["longest"])]
    A = s["A"].double()
    raw = s["dt"][0].double()
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"].double()
    step = torch.where(raw > 0, raw, 0.0) + torch.log1p(torch.exp(-raw.abs()))
    x = s["x"][0].double()
    spread = torch.arange(D, device=DEV) // (D // G)
    B, C = s["B"][0].double(), s["C"][0].double()
    h = torch.zeros(n, D, N, dtype=torch.float64, device=DEV)
    if s["init"] is not None:
        h += s["init"][order]
    u = torch.zeros(T, D, dtype=torch.float64, device=DEV)
    before = torch.empty(T, D, N, dtype=torch.float64, device=DEV) if c["train"] else None
    for t, m in enumerate(running):
        at = first[:m] + t
        if c["train"]:
            before[at] = h[:m]
        d = step[at]
        h[:m].mul_(torch.exp(d[..., None] * A)).add_((d * x[at])[..., None] * B[at][:, spread])
        u[at] = (h[:m] * C[at][:, spread]).sum(-1)
    back = torch.argsort(order)
    skip = s["D"].double() if s["D"] is not None else torch.zeros(D, device=DEV).double()
    u = u + skip * x
    gate = torch.ones_like(u)
    if s["z"] is not None:
        z = s["z"][0].double()
        gate = z / (1 + torch.exp(-z))
    out = [(u * gate)[None], h[back]]
    if not c["train"]:
        return out
    dy = s["dy"][0].double()
    du = dy * gate
    r = torch.zeros_like(h)
    if s["dfinal"] is not None:
        r += s["dfinal"][order]
    dA = torch.zeros_like(A)
    dB, dC = (torch.zeros(T, G, N, dtype=torch.float64, device=DEV) for _ in range(2))
    dx, dstep = torch.zeros_like(u), torch.zeros_like(u)
    for t in range(s["longest"] - 1, -1, -1):
        m = running[t]
        at = first[:m] + t
        d, xt, Bt = step[at], x[at], B[at][:, spread]
        a = torch.exp(d[..., None] * A)
        kept = before[at] * a
        dC[at] = (du[at][..., None] * (kept + (d * xt)[..., None] * Bt)).view(m, G, -1, N).sum(2)
        r[:m].add_(du[at][..., None] * C[at][:, spread])
        dB[at] = (r[:m] * (d * xt)[..., None]).view(m, G, -1, N).sum(2)
        inner = (r[:m] * Bt).sum(-1)
        kept *= r[:m]
        dx[at], dstep[at] = inner * d, inner * xt + (kept * A).sum(-1)
        dA += (kept * d[..., None]).sum(0)
        r[:m].mul_(a)
    ddt = dstep / (1 + torch.exp(-raw))
    out += [(dx + du * skip)[None], ddt[None], dA, dB[None], dC[None]]
    if s["D"] is not None:
        out.append((du * x).sum(0))
    if s["z"] is not None:
        sig = 1 / (1 + torch.exp(-z))
        out.append((dy * u * sig * (1 + z * (1 - sig)))[None])
    if s["dt_bias"] is not None:
        out.append(ddt.sum(0))
    if s["init"] is not None:
        out.append(r[back])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "conv":
        return _exact_conv(s)
    if op == "convstep":
        rows = [s["state"][:, k].double() for k in range(case["width"] - 1)] + [s["x"].double()]
        y = sum(r * s["weight"][:, k].double() for k, r in enumerate(rows))
        y = y if s["bias"] is None else y + s["bias"].double()
        return [y / (1 + torch.exp(-y)) if case["silu"] else y, torch.stack(rows[1:], 1)]
    if op == "scan":
        lens = _lens(case)
        cells, passes = case["dim"] * case["N"], 3 if case["train"] else 1
        if passes * (max(lens) * 150e-6 + sum(lens) * cells * 8 * 8 / 2e12) > 18 \
                or (case["train"] and sum(lens) * cells * 8 > 60e9):
            return None
        return _exact_scan(s)
    if op == "scanstep":
        c, D = case, case["dim"]
        raw = s["dt"].double() + (0.0 if s["dt_bias"] is None else s["dt_bias"].double())
        step = torch.where(raw > 0, raw, 0.0) + torch.log1p(torch.exp(-raw.abs()))
        spread = torch.arange(D, device=DEV) // (D // c["G"])
        h = s["state"].double() * torch.exp(step[..., None] * s["A"].double())
        h = h + (step * s["x"].double())[..., None] * s["B"].double()[:, spread]
        y = (h[:, :, None] @ s["C"].double()[:, spread][..., None])[..., 0, 0]
        y = y if s["D"] is None else y + s["D"].double() * s["x"].double()
        if s["z"] is not None:
            z = s["z"].double()
            y = y * z / (1 + torch.exp(-z))
        return [y, h]
    x, h = s["x"].double(), s["residual"].double()
    h = h + (x if s["scale"] is None else x * s["scale"].double())
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    y = y.unflatten(-1, (-1, case["group"]))
    top = CODES[case["code"]][1]
    scales = y.abs().amax(-1, keepdim=True) / top
    v = y / scales.clamp(min=1e-300)
    if case["code"] == "e4m3":
        # 4 significant bits, the smallest step 2^-9
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    else:
        unit = torch.ones_like(v)
    return [(torch.round(v / unit) * unit * scales).flatten(-2), scales[..., 0], h]
