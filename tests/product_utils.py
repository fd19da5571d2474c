"""Plain 64-bit forms of the packed product, its epilogue and the norm, for the
tests. Element values come from the format definitions; nothing here calls
the library."""
import numpy as np
import torch

DEV = torch.device("cuda:0")
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
ACTS = ("none", "gelu", "silu", "relu2", "swiglu")


def e4m3_table():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = -x if b & 128 else x
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = e4m3_table()


def unpack(q, K):
    """Packed codes [R, ceil(K/2)] -> E2M1 values [R, K]."""
    out = np.empty((q.shape[0], 2 * q.shape[1]))
    out[:, 0::2] = E2M1[q & 15]
    out[:, 1::2] = E2M1[q >> 4]
    return out[:, :K]


class Lines:
    """Packed lines on the host: u [R, K] values without the amax factor."""

    def __init__(self, q, s, amax, mode, bound, K):
        self.q, self.s, self.amax, self.mode, self.bound, self.K = q, s, amax, mode, bound, K
        R = q.shape[0]
        if s is None:
            self.u, f = E4M3[q], np.float64(np.float32(1) / np.float32(448))
        else:
            self.u = unpack(q, K) * np.repeat(E4M3[s], 16, 1)[:, :K]
            f = np.float64(np.float32(1) / (np.float32(bound) * np.float32(6)))
        self.line = np.broadcast_to(amax.astype(np.float64) * f, (R,))

    def dev(self, shift=0):
        """(q, s, amax) on the device; shift: bytes the packed data starts into its buffer."""
        def put(a):
            t = torch.empty(a.size + 64, dtype=torch.uint8, device=DEV)[shift:shift + a.size]
            t.copy_(torch.from_numpy(a.reshape(-1)))
            return t.view(*a.shape)
        q = put(self.q)
        if self.s is None:
            q = q.view(torch.float8_e4m3fn)
        return q, None if self.s is None else put(self.s), torch.from_numpy(self.amax).to(DEV)


def random_lines(rng, R, K, fmt="nvfp4", mode=1, bound=448.0, exact=False):
    """Random packed lines. exact: block scales 1 .. 8 (integers), 8-bit values
    -8 .. 8 (integers), amaxes powers of two and a bound whose factor is one:
    every product is a multiple of 1/4, so FP32 sums are exact in any order."""
    n = R if mode == 1 else 1
    if exact:
        bound = np.float32(512.0 / 6.0)
        assert np.float32(bound) * np.float32(6) == 512
    if fmt == "e4m3":
        if exact:
            q = (rng.randint(1, 9, (R, K)) * rng.choice([-1, 1], (R, K))).astype(np.float64)
            q = np.searchsorted(E4M3[:127], np.abs(q)).astype(np.uint8) | (128 * (q < 0)).astype(np.uint8)
        else:
            q = rng.randint(0, 127, (R, K)).astype(np.uint8) | (128 * rng.randint(0, 2, (R, K))).astype(np.uint8)
        s = None
    else:
        q = rng.randint(0, 256, (R, (K + 1) // 2)).astype(np.uint8)
        if K % 2:
            q[:, -1] &= 15
        nb = (K + 15) // 16
        if exact:
            s = np.searchsorted(E4M3[:127], rng.randint(1, 9, (R, nb)).astype(np.float64)).astype(np.uint8)
        else:
            s = rng.randint(0, 127, (R, nb)).astype(np.uint8)
    if exact:
        amax = np.float32(2.0) ** rng.randint(-3, 4, n).astype(np.float32)
        if fmt == "e4m3":
            amax = (amax * np.float32(448)).astype(np.float32)  # (a / 448 is rounded: see below)
    else:
        amax = np.exp(rng.uniform(-3, 3, n)).astype(np.float32)
    return Lines(q, s, amax.astype(np.float32), mode, float(bound), K)


def act64(act, z, N):
    if act == "gelu":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "relu2":
        return np.maximum(z, 0) ** 2
    if act == "swiglu":
        g = z[:, :N]
        return g / (1 + np.exp(-g)) * z[:, N:]
    return z


def dact64(act, dy, z, N):
    if act == "none":
        return dy
    if act == "relu2":
        return dy * 2 * np.maximum(z, 0)
    if act == "gelu":
        c = np.sqrt(2 / np.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    g = z[:, :N]
    s = 1 / (1 + np.exp(-g))
    ds = s * (1 + g * (1 - s))
    return dy * ds if act == "silu" else np.concatenate((dy * z[:, N:] * ds, dy * g * s), 1)


def np64(t):
    return t.detach().double().cpu().numpy()
