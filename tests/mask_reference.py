"""The dropout mask as factors of many rows at once, for sizes at which
norm_reference.keep takes too long: the same generator in torch's 64-bit
integers, on any device.  Products of two 32-bit words wrap modulo 2^64, which
leaves their low and (shifted, masked) high words right."""

from __future__ import annotations

import torch

from norm_reference import LOW, drop_count

M64 = (1 << 64) - 1


def keep(rows: int, cols: int, p: float, seed: int, offset: int, device="cpu", first: int = 0) -> torch.Tensor:
    """rows x cols factors in float64: 0 where dropped, 65536 / (65536 - drop) where kept.  `first`: the first row's first
    block, where it is not the matrix's."""
    drop = drop_count(p)
    if drop == 0:
        return torch.ones(rows, cols, dtype=torch.float64, device=device)
    each = -(-cols // 8)
    block = torch.arange(first, first + rows * each, dtype=torch.int64, device=device)
    place = offset & M64
    c = [block & LOW, block >> 32 & LOW, torch.full_like(block, place & LOW), torch.full_like(block, place >> 32)]
    k = [seed & LOW, seed >> 32]
    for _ in range(10):
        m0, m1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(m1 >> 32 & LOW) ^ c[1] ^ k[0], m1 & LOW, (m0 >> 32 & LOW) ^ c[3] ^ k[1], m0 & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    words = torch.stack(c, 1)
    numbers = torch.stack([words & 0xFFFF, words >> 16], 2).view(rows, each * 8)[:, :cols]
    scale = 65536 / (65536 - drop) if drop < 65536 else 0.0
    return torch.where(numbers < drop, 0.0, torch.tensor(scale, dtype=torch.float64, device=device))
