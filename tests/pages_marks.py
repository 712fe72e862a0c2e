"""Keys and values whose products say which positions of a history were summed, with which
key, value and bias.

Position i is marked with zeros and ones: column 0 is 1, columns 1 .. 20 are the bits of i,
the others bits of products of i.  With marks for keys and values, q = 64 in one column and
bias tables of 64 and 128 and of 0 and 64, a score is 64 to 256, SiLU of it is the score
itself in fp32 (exp(-64) is far below half a step of one), and every sum is a multiple of 64
below 2^24 * 64: exact in any order, so that one position too many, too few or with another
key is seen."""
import torch

SCORE = 64.0
BITS = 20


def marks(index: torch.Tensor, columns: int) -> torch.Tensor:
    """[..., columns] of the positions ``index`` (int64, below 2^20)."""
    c = torch.arange(columns, device=index.device)
    i = index[..., None]
    mixed = (i * (2 * c + 2654435761) >> 13) & 1
    bits = (i >> (c - 1).clamp(0, BITS)) & 1
    return torch.where(c == 0, torch.ones_like(mixed), torch.where(c <= BITS, bits, mixed))
