"""Packed rows in plain PyTorch, on any device: layouts, random rows, and what
rows stand for in 64 bits."""
import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Layout:
    """A packed row layout and the query heads that attend to it."""

    def __init__(self, heads, key, value, kv=1, wide=0, shared=False, dtype="bf16"):
        self.heads, self.key, self.value, self.kv = heads, key, value, kv
        self.wide, self.shared, self.dtype = wide, shared, dtype
        self.key8, self.scale = key - wide, key ** -0.5
        values = 0 if shared else kv * value
        self.off_value = kv * self.key8
        self.off_wide = self.off_value + values
        self.off_scale = self.off_wide + 2 * kv * wide
        self.scales = kv * (1 if shared else 2)
        self.row_bytes = -(-(self.off_scale + 4 * self.scales) // 16) * 16

    @property
    def type(self):
        return TYPES[self.dtype]

    def rows(self, dhs):
        return dhs.packed_rows(dtype=self.dtype, kv_heads=self.kv, key_elems=self.key,
                               wide_elems=self.wide, value_elems=self.value, shared=self.shared)

    def assemble(self, key, value, wide, scales):
        """Rows [n, bytes] of codes (uint8 [n, kv, .]), 16-bit elements and scales."""
        n, dev = len(key), key.device
        parts = [key.reshape(n, -1)]
        if not self.shared:
            parts.append(value.reshape(n, -1))
        if self.wide:
            parts.append(wide.to(self.type).contiguous().view(torch.uint8).reshape(n, -1))
        parts.append(scales.float().contiguous().view(torch.uint8).reshape(n, -1))
        pad = self.row_bytes - self.off_scale - 4 * self.scales
        return torch.cat(parts + [torch.zeros(n, pad, dtype=torch.uint8, device=dev)], 1)

    def random(self, n, g, low=-3, high=3):
        """n rows of random codes (no NaN) and scales 2^low .. 2^high."""
        dev = g.device
        code = lambda m: (torch.randn(n, self.kv, m, generator=g, device=dev) * 40).clamp(-448, 448) \
            .to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        e = torch.randint(low, high + 1, (n, self.scales), generator=g, device=dev) - 5
        wide = torch.randn(n, self.kv, self.wide, generator=g, device=dev)
        return self.assemble(code(self.key8), code(self.value), wide, torch.exp2(e.float()))

    def numbers(self, rows):
        """Keys [n, kv, key] and values [n, kv, value] in 64 bits."""
        n, kv = len(rows), self.kv
        part = lambda a, m, t: rows[:, a:a + m].contiguous().view(t).double()  # noqa: E731
        scale = part(self.off_scale, 4 * self.scales, torch.float32).view(n, self.scales // kv, kv)
        key = part(0, kv * self.key8, torch.float8_e4m3fn).view(n, kv, self.key8) * scale[:, 0, :, None]
        if self.shared:
            value = key[..., :self.value]
        else:
            value = part(self.off_value, kv * self.value, torch.float8_e4m3fn).view(n, kv, self.value) * \
                scale[:, 1, :, None]
        if self.wide:
            key = torch.cat([key, part(self.off_wide, 2 * kv * self.wide, self.type).view(n, kv, self.wide)], -1)
        return key, value


LAYOUTS = {
    "latent": Layout(16, 576, 512, wide=64, shared=True),
    "latent_f16": Layout(24, 576, 512, wide=64, shared=True, dtype="f16"),
    "latent_one_head": Layout(1, 576, 512, wide=64, shared=True),
    "latent_40": Layout(40, 576, 512, wide=64, shared=True),
    "latent_64": Layout(64, 576, 512, wide=64, shared=True),
    "latent_64_f16": Layout(64, 576, 512, wide=64, shared=True, dtype="f16"),
    "latent_100": Layout(100, 576, 512, wide=64, shared=True),
    "latent_128": Layout(128, 576, 512, wide=64, shared=True),
    "grouped": Layout(40, 128, 128, kv=8),
    "grouped_f16": Layout(6, 96, 64, kv=2, dtype="f16"),
    "grouped_wide": Layout(32, 192, 128, kv=4, wide=64),
    "grouped_some_wide": Layout(8, 64, 192, kv=4, wide=16, dtype="f16"),
    "smallest": Layout(3, 16, 16),
    "odd": Layout(17, 80, 48, wide=32),
    "same": Layout(33, 64, 64, shared=True),
    "part_of_key": Layout(12, 160, 80, kv=2, shared=True),
    "no_wide": Layout(20, 576, 512),
    "no_wide_f16": Layout(48, 576, 512, dtype="f16"),
    "no_wide_64": Layout(64, 576, 512),
    "wide_eight": Layout(5, 200, 208, wide=8),
}


def exponent(top):
    """The smallest e in [-64, 120] with top <= 448 * 2^e."""
    if top == 0:
        return -64
    m, x = math.frexp(top)
    return max(-64, min(120, x - (9 if m <= 0.875 else 8)))


def codes_of(x):
    """The codes (uint8) and scales of heads x [..., n] in 64 bits, by the rule:
    the power of two from the largest finite element, each element to the
    nearest code with ties to even, NaN for what is not finite."""
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0).amax(-1)
    e = torch.tensor([exponent(t) for t in top.reshape(-1).tolist()], dtype=torch.float64,
                     device=x.device).view(top.shape)
    scale = torch.exp2(e)
    every = torch.arange(127, device=x.device)  # the codes of the numbers from 0 up
    value = every.to(torch.uint8).view(torch.float8_e4m3fn).double()
    y = (torch.where(fine, x, 0) / scale[..., None]).abs()
    hi = torch.searchsorted(value, y.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = value[hi] - y, y - value[lo]
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(torch.signbit(torch.where(fine, x, 0)), code + 128, code)
    return torch.where(fine, code, 127).to(torch.uint8), scale
