"""64-bit references of the norm and the dense product in 8 bits, and their error bounds."""
import torch

U = 2.0 ** -24  # a rounding to fp32, relative to the value


def blocks(x):
    """x [n][d] in blocks of 128 columns, the last one filled up with zeros: [n][blocks][128]."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 128)).unflatten(1, (-1, 128))


def decode(q, s):
    """fp64 values of E4M3 codes with a scale per 128 columns."""
    return (blocks(q.float().double()) * s.double()[:, :-(-q.shape[1] // 128), None]).flatten(1)[:, :q.shape[1]]


def grid(device):
    """All finite E4M3 values, ascending."""
    v = torch.arange(256, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn).double()
    return v[v.isfinite()].unique()


def distance(u):
    """Distance of each value (fp64) to the nearest E4M3 value."""
    g = grid(u.device)
    at = torch.searchsorted(g, u.contiguous()).clamp(1, g.numel() - 1)
    return torch.minimum((u - g[at - 1]).abs(), (u - g[at]).abs())


def weights(N, K, g, device="cuda"):
    """E4M3 weights [N][K] and fp32 scales per 128 x 128 block."""
    w = torch.randn(N, K, device=device, generator=g) * K ** -0.5
    full = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128)).view(-(-N // 128), 128, -(-K // 128), 128)
    s = full.abs().amax((1, 3)) / 448
    q = (full / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(-(-N // 128) * 128, -1)[:N, :K].contiguous(), s.contiguous()


def quantised(T, K, g, device="cuda"):
    """E4M3 rows [T][K] and fp32 scales per 128 columns."""
    x = blocks(torch.randn(T, K, device=device, generator=g) * torch.exp(0.4 * torch.randn(K, device=device, generator=g)))
    s = (x.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    return (x / s[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(1)[:, :K].contiguous(), s


def product(xq, xs, wq, ws):
    """The product in 64 bits, and the sum of the magnitudes of its terms."""
    x = decode(xq, xs)
    w = (blocks(wq.float().double()) * ws.double().repeat_interleave(128, 0)[:wq.shape[0], :, None]).flatten(1)[:, :wq.shape[1]]
    return x @ w.T, x.abs() @ w.abs().T


def bound(ref, mag, K, dtype):
    """How far an output may be off. Products of codes are exact. A block's sum takes four matrix
    instructions, each of which may truncate once (2 U of the terms' magnitude); the block's scale is
    a product of two (one rounding) and every block adds with one: (8 + 1 + blocks) U of the sum of
    magnitudes; the output is rounded once."""
    fp32 = (9 + -(-K // 128)) * U * mag
    half = torch.finfo(dtype).eps / 2
    return fp32 * (1 + half) + half * ref.abs() + 1e-38
