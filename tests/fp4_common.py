"""4-bit codes and block scales in 64 bits, for the tests of the 4-bit quantisation and products."""
import torch

BLOCK = {"nvfp4": 16, "mxfp4": 32}
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e2m1_values(packed):
    """[rows, K/2] bytes -> [rows, K] values."""
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=packed.device)
    return table[torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1).long()]


def scale_values(byte, fmt):
    return byte.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.exp2(byte.double() - 127.0)


def tiled(scale, fill):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 scales, the padding filled with `fill`."""
    rows, blocks = scale.shape
    full = torch.full(((rows + 127) // 128 * 128, (blocks + 3) // 4 * 4), fill, dtype=torch.uint8, device=scale.device)
    full[:rows, :blocks] = scale
    return full.reshape(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def untiled(tiles, rows, blocks):
    """(scale bytes [rows, blocks], the padding's bytes)."""
    wide = (blocks + 3) // 4
    full = tiles.reshape(-1, wide, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * wide)
    pad = torch.ones_like(full, dtype=torch.bool)
    pad[:rows, :blocks] = False
    return full[:rows, :blocks].contiguous(), full[pad]


def decoded(packed, scale, fmt):
    """Codes and row-major scale bytes -> [rows, K] values in 64 bits."""
    v = e2m1_values(packed).unflatten(1, (-1, BLOCK[fmt]))
    return (v * scale_values(scale, fmt)[:, :, None]).flatten(1)


def nearest(t):
    """E2M1 value nearest to t, ties to the even code."""
    a, value = t.abs(), torch.zeros_like(t)
    for i, (low, high) in enumerate(zip(VALUES, VALUES[1:])):
        mid = (low + high) / 2
        value += (high - low) * ((a >= mid) if i % 2 else (a > mid))
    return torch.copysign(value, t)
