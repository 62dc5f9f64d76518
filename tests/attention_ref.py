"""Float64 reference of the attention calls with a relative position bias, and
elementwise bounds on what a correct float32-accumulating kernel may be off.

Bounds.  u = eps / 2 of the storage type is the half step of one rounding
(0 for float32, whose kernels round no operand); w = 2^-23 is one float32
rounding or truncation of a sum.  With X the scores,
  |dx|   <= (d + 8) w (c |Q||K|^T + |bias| + |mask| + |lse|)
            (d products and sums, then scale, bias, mask, reference in log2 units)
  |dP|/P <= e := |dx| + 8 w                              (base-2 exponential, sum)
  O:  P rounded (u), the sum over the keys (e and S w at most, the terms'
      order unknown), O rounded (u):   (u + 2 e + S w) P|V| + u |O|
  dV: (u + e + S w) P^T|dO| + u |dV|
  dS: P (dP - D):  E := (e + (d + 4) w) P (|dO||V|^T + |dO|.|O|)
  dQ: c ((u + S w) |dS| |K| + E |K|) + u |dQ|, dK alike, dT: E + S B w |dS| summed.
float16 keeps an operand below 2^-14 to an absolute 2^-25 only: P and dS gain
that much per entry.
"""
import math

import torch

MASKED = -1e30
W = 2.0 ** -23


def bucket(rel: int, buckets: int, distance: int) -> int:
    """Bucket of key minus query position, in whole numbers."""
    side, n = (buckets // 2 if rel > 0 else 0), abs(rel)
    half, first = buckets // 2, buckets // 4
    if n < first:
        return side + n
    steps, k = half - first, 0
    while k + 1 < steps and n ** steps >= first ** (steps - k - 1) * distance ** (k + 1):
        k += 1
    return side + first + k


def bucket_matrix(s: int, buckets: int, distance: int, device) -> torch.Tensor:
    ids = torch.tensor([bucket(r, buckets, distance) for r in range(-(s - 1), s)], device=device)
    pos = torch.arange(s, device=device)
    return ids[pos[None, :] - pos[:, None] + s - 1]


def bias_of(table, s, distance):
    ids = bucket_matrix(s, table.shape[0], distance, table.device)
    return table.double().t()[:, ids], ids            # (heads, s, s)


def scores(q, k, mask, table, distance, scale):
    q, k = q.double().transpose(1, 2), k.double().transpose(1, 2)
    x = scale * q @ k.transpose(2, 3)
    size = scale * q.abs() @ k.abs().transpose(2, 3)
    if table is not None:
        bias, _ = bias_of(table, q.shape[2], distance)
        x = x + bias
        size = size + bias.abs()
    if mask is not None:
        m = mask.double()[:, None, None]
        gone = (m <= MASKED).expand_as(x)
        x = torch.where(gone, -math.inf, x + m)
        size = torch.where(gone, 0.0, size + m.abs())
    return x, size


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def half_step(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def forward(q, k, v, mask=None, table=None, distance=128, scale=None):
    """({name: value}, {name: bound}) for o and lse."""
    d, s = q.shape[3], q.shape[1]
    scale = d ** -0.5 if scale is None else scale
    x, size = scores(q, k, mask, table, distance, scale)
    lse = torch.logsumexp(x, -1)
    empty = lse == -math.inf
    p = torch.exp(x - torch.where(empty, 0.0, lse)[..., None])
    vv = v.double().transpose(1, 2)
    o = p @ vv
    u, w = half_step(q.dtype), W
    e = (d + 8) * w * (size + torch.where(empty, 0.0, lse).abs()[..., None]) + 8 * w
    o_tol = ((p * (u + 2 * e + s * w)) @ vv.abs() + u * o.abs() + tiny(q.dtype) * (p > 0).double() @ vv.abs() + 2 * w * o.abs()
             + torch.finfo(q.dtype).tiny)
    lse_tol = (p * e).sum(-1) + (s + 8) * w + 4 * w * torch.where(empty, 0.0, lse).abs()
    return ({"o": o.transpose(1, 2), "lse": torch.where(empty, math.inf, lse)},
            {"o": o_tol.transpose(1, 2), "lse": lse_tol})


def backward(q, k, v, o, lse, do, mask=None, table=None, distance=128, scale=None):
    d, s, b = q.shape[3], q.shape[1], q.shape[0]
    scale = d ** -0.5 if scale is None else scale
    x, size = scores(q, k, mask, table, distance, scale)
    lse = lse.double()
    p = torch.exp(x - lse[..., None])
    qq, kk, vv, oo, dd = (t.double().transpose(1, 2) for t in (q, k, v, o, do))
    delta = (dd * oo).sum(-1, keepdim=True)
    ds = p * (dd @ vv.transpose(2, 3) - delta)
    val = {"dq": scale * ds @ kk, "dk": scale * ds.transpose(2, 3) @ qq, "dv": p.transpose(2, 3) @ dd}
    u, w, t = half_step(q.dtype), W, tiny(q.dtype)
    lf = torch.where(lse == math.inf, 0.0, lse)
    e = (d + 8) * w * (size + lf.abs()[..., None]) + 8 * w
    err = (e + (d + 4) * w) * p * (dd.abs() @ vv.abs().transpose(2, 3) + (dd.abs() * oo.abs()).sum(-1, keepdim=True))
    on = (p > 0).double()
    own = (u + s * w) * ds.abs() + err + t * on
    tol = {"dq": scale * own @ kk.abs(), "dk": scale * own.transpose(2, 3) @ qq.abs(),
           "dv": ((u + e + s * w) * p + t * on).transpose(2, 3) @ dd.abs()}
    tol = {n: tol[n] + (u + 2 * w) * val[n].abs() + torch.finfo(q.dtype).tiny for n in tol}
    val, tol = ({n: x.transpose(1, 2) for n, x in y.items()} for y in (val, tol))
    if table is not None:
        ids = bucket_matrix(s, table.shape[0], distance, q.device).reshape(-1)
        every = ((err + (s * b + 8) * w * ds.abs()).sum(0), ds.sum(0))
        got = [torch.zeros(table.shape[0], q.shape[2], dtype=torch.float64, device=q.device)
               .index_add_(0, ids, z.reshape(q.shape[2], -1).t()) for z in every]
        val["dtable"], tol["dtable"] = got[1], got[0] + 4 * w * got[1].abs() + 1e-30
    return val, tol
