"""Plain 64-bit forms of the training operators, for the tests: numpy or
float64 torch on the CPU, written from the formulas of include/gcq.h."""
import numpy as np
import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# what a value may be off by where it rounds to a subnormal or to zero
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in HALF_STEP}
F32 = 2.0 ** -24


def philox(slots: np.ndarray, seed: int, worker: int, purpose: int) -> np.ndarray:
    """[len(slots), 4] words of Philox4x32-10 at the counters (slot low, slot
    high, worker, purpose)."""
    m, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    slots = np.asarray(slots, np.uint64)
    c = [slots & m, slots >> sh, np.full_like(slots, worker), np.full_like(slots, purpose)]
    k = [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1).astype(np.uint32)


def keep(n: int, p: float, seed: int, worker: int, offset: int = 0) -> np.ndarray:
    """Whether values offset .. offset + n - 1 of the mask are kept."""
    first = offset >> 2
    slots = np.array([first + k for k in range(((offset & 3) + n + 3) // 4)], dtype=np.uint64)
    r = philox(slots, seed & (2 ** 64 - 1), worker, 2).reshape(-1)[offset & 3:][:n]
    return (r >> 8).astype(np.float64) * 2.0 ** -24 >= p


def factor(n: int, p: float, seed: int, worker: int, offset: int = 0) -> torch.Tensor:
    """0 where dropped, 1 / (1 - p) where kept, float64."""
    if p >= 1.0:
        return torch.zeros(n, dtype=torch.float64)
    return torch.from_numpy(keep(n, p, seed, worker, offset).astype(np.float64) / (1.0 - p))
