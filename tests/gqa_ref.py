"""Plain fp64 restatements of the operators for layers whose heads keep their own keys and
values, with the sizes their error bounds need.  Test infrastructure only."""
import math

import torch

F32 = 2.0 ** -24          # half a step of fp32, relative
BF16 = 2.0 ** -8
F16 = 2.0 ** -11
E4M3 = 2.0 ** -4


def rotate(x, cos_sin, positions, neox):
    """(value, magnitude) in fp64: x (T, H, D) with its first R columns turned; magnitude =
    |x cos| + |y sin|, what the fp32 products can be off by in units of 2^-24."""
    x = x.double()
    r = cos_sin.shape[1]
    row = cos_sin.double()[positions.long()][:, None, :]
    c, s = row[..., :r // 2], row[..., r // 2:]
    i = torch.arange(r // 2, device=x.device)
    a, b = (i, i + r // 2) if neox else (2 * i, 2 * i + 1)
    out, mag = x.clone(), x.abs()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return out, mag


def attend(q, k, v, scale, limit):
    """One KV head: q (n, d), k (m, d), v (m, dv) fp64, row i sees keys j < limit[i].
    Returns o, lse, mass = sum p |v| (what rounding the weights can move) and the largest
    score magnitude sum |q k| scale of each row."""
    n, m = q.shape[0], k.shape[0]
    if m == 0:
        z = torch.zeros(n, v.shape[1], dtype=torch.float64, device=q.device)
        return z, torch.full((n,), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    s = (q @ k.T) * scale
    seen = torch.arange(m, device=q.device)[None, :] < limit[:, None]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, dim=1)
    p = torch.where(seen, torch.exp(s - lse[:, None].clamp_min(-1e300)), torch.zeros_like(s))
    big = torch.where(seen, (q.abs() @ k.abs().T) * abs(scale), torch.zeros_like(s)).amax(dim=1)
    vv = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
    return p @ vv, lse, p @ vv.abs(), big


def bounds(o, lse, mass, big, n_keys, d, weight_eps, out_eps):
    """Allowed |o - o_ref| and |lse - lse_ref|.

    A score is a sum of d exact products in fp32 and two multiplications: off by at most
    (d + 2) 2^-24 big; its exponential by as much relative, twice 2^-22 more for exp2 and
    its argument's rounding (|argument| up to 1.45 big).  The same error in every weight of
    the numerator and of the sum gives 2x; sums over n_keys terms in fp32 add n_keys 2^-24
    each, the online rescaling 2^-22 a tile at most.  The weights are rounded by weight_eps
    in the numerator only, the result by out_eps.
    """
    ds = ((d + 2) + 4) * F32 * big + 2.0 ** -21
    rel = 2 * ds + 2 * n_keys * F32 + (n_keys / 16 + 64) * 2.0 ** -22
    ob = out_eps * o.abs() + (1 + out_eps) * (weight_eps + rel[..., None]) * mass + 1e-30
    lb = ds + n_keys * F32 + (n_keys / 16 + 64) * 2.0 ** -22 + 4 * F32 * (lse.abs() + big) + 2.0 ** -20
    return ob, lb


def check(got_o, got_lse, ref, n_keys, d, weight_eps, out_eps, what=""):
    """got against ref = (o, lse, mass, big), rows with lse = -inf exactly."""
    o, lse, mass, big = ref
    empty = torch.isneginf(lse)
    ob, lb = bounds(o, torch.where(empty, torch.zeros_like(lse), lse), mass, big, n_keys, d,
                    weight_eps, out_eps)
    g = got_o.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    worst = ((g - o).abs() / ob).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: o error {worst:.3f} of its bound"
    assert (g[empty] == 0).all(), f"{what}: an empty row is not zero"
    if got_lse is not None:
        gl = got_lse.double()
        assert torch.equal(torch.isneginf(gl), empty), f"{what}: lse of empty rows"
        d_l = torch.where(empty, torch.zeros_like(gl), (gl - lse).abs())
        worst_l = (d_l / lb).max().item() if gl.numel() else 0.0
        assert worst_l <= 1.0, f"{what}: lse error {worst_l:.3f} of its bound"
    return worst
