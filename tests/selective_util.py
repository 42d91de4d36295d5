"""Inputs, packing and guarded outputs of the selective operators' GPU tests."""
import math
import random

import torch

DEV = "cuda:0"
GUARD = 256
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


class Guarded:
    """Tensors with GUARD bytes of a pattern on either side; NaN bytes inside."""

    def __init__(self):
        self.buffers = []

    def __call__(self, shape, dtype):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        pad = -n % 16
        buf = torch.full((n + pad + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
        buf[GUARD:GUARD + n] = 0xFF
        self.buffers.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        for buf, n in self.buffers:
            assert (buf[:GUARD] == 0xA5).all() and (buf[GUARD + n:] == 0xA5).all()


def spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw_lens(rng, total, packed):
    """Lengths, and rows before and behind the sequences."""
    if not packed:
        n = rng.choice([1, 2, 5])
        return {"lens": [max(1, total // n)] * n, "before": 0, "after": 0}
    lens, left = [], total
    for _ in range(rng.choice([0, 1, 3, 9])):
        lens.append(rng.randint(0, left))
        left -= lens[-1]
    return {"lens": lens + [left], "before": rng.choice([0, 0, 3]),
            "after": rng.choice([0, 0, 70])}


class Rows:
    """Random rows [rows, *shape] on the device, NaN outside the sequences, as columns of
    a wider tensor where `wide`; `cut` gives those of the sequences in 64 bits."""

    def __init__(self, c, seed):
        self.c, self.g = c, torch.Generator().manual_seed(seed)
        self.T = sum(c["lens"])
        self.rows = self.T + c["before"] + c["after"]
        self.at = slice(c["before"], c["before"] + self.T)
        self.lead = (1, self.rows) if c["packed"] else (len(c["lens"]), c["lens"][0])
        self.cu = None
        if c["packed"]:
            ends = [c["before"]]
            for n in c["lens"]:
                ends.append(ends[-1] + n)
            self.cu = torch.tensor(ends, dtype=torch.int32, device=DEV)

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=self.g) * std).to(dtype)

    def __call__(self, *shape, dtype, std=1.0, offset=0.0, wide=False):
        t = (torch.randn(self.rows, *shape, generator=self.g) * std + offset).to(dtype)
        t[:self.at.start] = float("nan")
        t[self.at.stop:] = float("nan")
        dev = t.to(DEV).view(*self.lead, *shape)
        if wide:
            n = math.prod(shape)
            buf = torch.full((*self.lead, n + 24), float("nan"), dtype=dtype, device=DEV)
            buf[..., 8:8 + n] = dev.flatten(len(self.lead))
            dev = buf[..., 8:8 + n].unflatten(-1, shape)
        return dev, t[self.at].double()

    def cut(self, name, t):
        """A row result: the sequences' rows; those outside were left alone."""
        t = t.reshape(self.rows, *t.shape[2:])
        assert torch.isnan(torch.cat([t[:self.at.start], t[self.at.stop:]])).all(), name
        return t[self.at]


def dev(t):
    return None if t is None else t.to(DEV)


def dbl(t):
    return None if t is None else t.double().cpu()


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def name_of(c):
    return "_".join(f"{k[:2]}{v}" for k, v in c.items()).replace(" ", "")[:90]


def rng_of(seed):
    return random.Random(seed)
