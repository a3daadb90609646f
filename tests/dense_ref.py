"""References for the dense operators in 64 bits, on whatever device the inputs are, and
the sums of magnitudes that their tolerances count."""
import torch

IGNORE = -100


def loss(x, weight, target, ignore=IGNORE):
    """(loss, lse, p) of softmax cross entropy, row by row; ignored rows zero.  Their x
    is not read."""
    x = torch.where((target != ignore)[:, None], x, 0).double()
    z = x @ weight.double().T
    lse = z.logsumexp(1)
    at = torch.where(target == ignore, 0, target)[:, None]
    row = torch.where(target == ignore, 0.0, lse - z.gather(1, at)[:, 0])
    return row, lse, (z - lse[:, None]).exp()


def loss_gradient(x, weight, target, g, ignore=IGNORE):
    """(dx, dweight) for upstream gradients g [rows], and for each the sum over its terms'
    magnitudes: |dz| |weight|, |dz|^T |x|."""
    kept = target != ignore
    _, _, p = loss(x, weight, target, ignore)
    dz = p.clone()
    dz.scatter_add_(1, torch.where(kept, target, 0)[:, None], torch.full_like(p[:, :1], -1.0))
    dz = torch.where(kept[:, None], dz * g.double()[:, None], 0)
    x = torch.where(kept[:, None], x, 0).double()
    w = weight.double()
    return dz @ w, dz.T @ x, dz.abs() @ w.abs(), dz.abs().T @ x.abs()


def values(codes, scales, blocks=False):
    """What an 8-bit matrix with groups (blocks) of 128 stands for."""
    rows = torch.arange(codes.shape[0], device=codes.device) // (128 if blocks else 1)
    cols = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.float().double() * scales.double()[rows][:, cols]


def pack_blocks(w):
    """(codes, scales) of a matrix with one scale per 128 x 128 block, in fp32 steps (they
    are defined bit for bit)."""
    w = w.float()
    rows, cols = w.shape
    codes = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty(-(-rows // 128), -(-cols // 128), device=w.device)
    top = torch.tensor(448.0, device=w.device)
    for r in range(0, rows, 128):
        for c in range(0, cols, 128):
            part = w[r:r + 128, c:c + 128]
            m = part.abs().max() if not part.isnan().any() else torch.tensor(float("nan"), device=w.device)
            if not torch.isfinite(m):
                scale, inverse = torch.full_like(m, float("nan")), torch.zeros_like(m)
            elif m < 2.0 ** -100:
                scale, inverse = torch.zeros_like(m), torch.zeros_like(m)
            else:
                scale, inverse = m / top, top / m
            scales[r // 128, c // 128] = scale
            part = torch.nan_to_num(part, 0, 0, 0) * inverse if inverse > 0 else torch.zeros_like(part)
            codes[r:r + 128, c:c + 128] = part.clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, scales
