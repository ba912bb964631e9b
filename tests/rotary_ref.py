"""Plain 64-bit reference of the rotation (CPU, torch double), written from its definition."""
import torch


def turns(positions, inv_freq, axis, axes):
    """e^(i theta) [tokens, pairs]; a pair on no axis stands at position 0. The product of a position below 2^26
    and a frequency is rounded in 64 bits, by more than the kernel's angle is off; so the frequency is taken in
    two parts of 27 and 26 bits, whose products are exact, and their turns are multiplied."""
    p = positions.view(1, -1) if positions.dim() == 1 else positions
    assert p.abs().max() < 1 << 26
    out = torch.ones(p.shape[1], inv_freq.numel(), dtype=torch.complex128)
    for i, w in enumerate(inv_freq.tolist()):
        a = int(axis[i]) if axis is not None else 0
        if 0 <= a < axes:
            high = w * (2.0 ** 26 + 1) - (w * (2.0 ** 26 + 1) - w)
            t = p[a].double()
            for part in (high, w - high):
                out[:, i] *= torch.polar(torch.ones_like(t), t * part)
    return out


def pairs_of(x, pairs, adjacent):
    return (x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]) if adjacent else (x[..., :pairs], x[..., pairs:2 * pairs])


def put_pairs(x, a, b, pairs, adjacent):
    y = x.clone()
    if adjacent:
        y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2] = a, b
    else:
        y[..., :pairs], y[..., pairs:2 * pairs] = a, b
    return y


def rotate(x, turn, adjacent, factor=1.0, transpose=False):
    """The turned rows, and the bound of an fp32 evaluation: c and s are each off by half a step, and so are
    the two products and their sum: |x0 c| + |x1 s| times 2 half steps of 2^-24, and the sum's own. Second
    orders: 1 %. The smallest normal number covers steps of subnormal products."""
    P = turn.shape[1]
    x = x.double()
    c = (turn.real * factor).unsqueeze(1)
    s = (turn.imag * factor).unsqueeze(1) * (-1 if transpose else 1)
    a, b = pairs_of(x, P, adjacent)
    y, z = a * c - b * s, b * c + a * s
    ty = 1.01 * ((a * c).abs() + (b * s).abs()) * 2.0 ** -23 + y.abs() * 2.0 ** -24 + 2.0 ** -126
    tz = 1.01 * ((b * c).abs() + (a * s).abs()) * 2.0 ** -23 + z.abs() * 2.0 ** -24 + 2.0 ** -126
    return put_pairs(x, y, z, P, adjacent), put_pairs(torch.zeros_like(x), ty, tz, P, adjacent)


def rounded(x, turn, adjacent, factor=1.0, transpose=False):
    """The fp32 values bit for bit: c and s rounded from 64 bits, products and sum rounded one by one."""
    P = turn.shape[1]
    x = x.float()
    c = (turn.real * factor).float().unsqueeze(1)
    s = (turn.imag * factor).float().unsqueeze(1) * (-1 if transpose else 1)
    a, b = pairs_of(x, P, adjacent)
    return put_pairs(x, a * c - b * s, b * c + a * s, P, adjacent)


def within(got, want, tol):
    """got (bf16 or fp32) against 64 bits: bf16 adds half a step of the value it rounds."""
    if got.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all()
    assert (err <= tol).all(), ((err - tol).max().item(), err.max().item())
