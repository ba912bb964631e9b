"""Plain 64-bit reference of the rotation (CPU, torch double), written from its definition."""
import torch


def angles(positions, inv_freq, axis, axes):
    """[tokens, pairs]; a pair on no axis stands at position 0."""
    p = positions.view(1, -1) if positions.dim() == 1 else positions
    out = torch.zeros(p.shape[1], inv_freq.numel(), dtype=torch.float64)
    for i, w in enumerate(inv_freq.tolist()):
        a = int(axis[i]) if axis is not None else 0
        if 0 <= a < axes:
            out[:, i] = p[a].double() * w
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


def rotate(x, theta, adjacent, factor=1.0, transpose=False):
    """The turned rows, and the bound of an fp32 evaluation: c and s are each off by half a step, and so are
    the two products and their sum: |x0 c| + |x1 s| times 2 half steps of 2^-24, and the sum's own. Second
    orders: 1 %. The smallest normal number covers steps of subnormal products."""
    P = theta.shape[1]
    x = x.double()
    c = (torch.cos(theta) * factor).unsqueeze(1)
    s = (torch.sin(theta) * factor).unsqueeze(1) * (-1 if transpose else 1)
    a, b = pairs_of(x, P, adjacent)
    y, z = a * c - b * s, b * c + a * s
    ty = 1.01 * ((a * c).abs() + (b * s).abs()) * 2.0 ** -23 + y.abs() * 2.0 ** -24 + 2.0 ** -126
    tz = 1.01 * ((b * c).abs() + (a * s).abs()) * 2.0 ** -23 + z.abs() * 2.0 ** -24 + 2.0 ** -126
    return put_pairs(x, y, z, P, adjacent), put_pairs(torch.zeros_like(x), ty, tz, P, adjacent)


def rounded(x, theta, adjacent, factor=1.0, transpose=False):
    """The fp32 values bit for bit: c and s rounded from 64 bits, products and sum rounded one by one."""
    P = theta.shape[1]
    x = x.float()
    c = (torch.cos(theta) * factor).float().unsqueeze(1)
    s = (torch.sin(theta) * factor).float().unsqueeze(1) * (-1 if transpose else 1)
    a, b = pairs_of(x, P, adjacent)
    return put_pairs(x, a * c - b * s, b * c + a * s, P, adjacent)


def within(got, want, tol):
    """got (bf16 or fp32) against 64 bits: bf16 adds half a step of the value it rounds."""
    if got.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all()
    assert (err <= tol).all(), ((err - tol).max().item(), err.max().item())
