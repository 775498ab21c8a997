"""The paged operators restated in 64 bits on the CPU, with bounds on what
their rounding may move (plain loops, no code of the library)."""
import math

import torch

BF16_HALF = 2.0 ** -8      # half a step of bf16, relative to the value
F32_HALF = 2.0 ** -24
# A score is a sum of 576 products of bf16 values (exact in fp32): every
# addition moves it by at most a step of fp32 (2^-23, whatever the rounding) of
# the sum of magnitudes, and at most 576 of them follow one another.
SCORE_STEPS = 576


def slots_of(table_row, page, lo, hi):
    """Row numbers in the flat cache of positions lo..hi-1 of one request."""
    return torch.tensor([int(table_row[j // page]) * page + j % page for j in range(lo, hi)], dtype=torch.int64)


def rotate(x, ang, halves):
    """x [..., 64], ang [..., 64] = cos | sin, both fp64."""
    c, s = ang[..., :32], ang[..., 32:]
    y = torch.empty_like(x)
    one = slice(0, 32) if halves else slice(0, 64, 2)
    two = slice(32, 64) if halves else slice(1, 64, 2)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def append(latent, k_rope, indptr, lens, table, flat, page, rope_table, q_rope=None, positions=None,
           weight=None, eps=1e-6, halves=False):
    """(slots [T'], rows [T', 576], row bounds, q [T', H, 64], q bounds) for the
    tokens of all requests in order; all fp64 on the CPU."""
    slots, rows, rtol, qs, qtol = [], [], [], [], []
    for b in range(len(lens)):
        t0, t1 = int(indptr[b]), int(indptr[b + 1])
        n, le = t1 - t0, int(lens[b])
        if n == 0:
            continue
        slots.append(slots_of(table[b], page, le - n, le))
        pos = torch.arange(le - n, le) if positions is None else positions[t0:t1].long()
        ang = rope_table[pos].double()
        lat = latent[t0:t1].double()
        lt = torch.zeros_like(lat)
        if weight is not None:
            lat = lat / torch.sqrt((lat * lat).mean(-1, keepdim=True) + eps) * weight.double()
            # 512 squares summed, a quotient, a root and two products in fp32
            lt = lat.abs() * (BF16_HALF + 600 * F32_HALF)
        k = k_rope[t0:t1].double()
        kt = rotate(k, ang, halves)
        rows.append(torch.cat([lat, kt], 1))
        rtol.append(torch.cat([lt, _turn_tol(k, kt, halves)], 1))
        if q_rope is not None:
            x = q_rope[t0:t1].double()
            y = rotate(x, ang[:, None], halves)
            qs.append(y)
            qtol.append(_turn_tol(x, y, halves))
    cat = lambda v: torch.cat(v) if v else None  # noqa: E731
    return cat(slots), cat(rows), cat(rtol), cat(qs), cat(qtol)


def _turn_tol(x, y, halves):
    """Two fp32 products and their sum (each off by half a step of at most
    |x_a| + |x_b|, angles' sines and cosines being at most 1), then bf16."""
    if halves:
        s = x[..., :32].abs() + x[..., 32:].abs()
        s = torch.cat([s, s], -1)
    else:
        s = (x[..., 0::2].abs() + x[..., 1::2].abs()).repeat_interleave(2, -1)
    return y.abs() * BF16_HALF + 4 * F32_HALF * s


def decode(q, flat, table, lens, page, scale, bad_pages=()):
    """(out, lse, out bounds, lse bounds): q [B, H, 576] and flat [rows, 576]
    CPU tensors; positions in bad_pages are left out."""
    B, H, _ = q.shape
    out = torch.zeros(B, H, 512, dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    otol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        ids = [int(table[b][j // page]) * page + j % page for j in range(int(lens[b]))
               if int(table[b][j // page]) not in bad_pages]
        if not ids:
            continue
        k = flat[torch.tensor(ids, dtype=torch.int64)].double()
        x = q[b].double()
        s = (x @ k.T) * scale
        lse[b] = torch.logsumexp(s, -1)
        w = torch.exp(s - lse[b][:, None])
        v = k[:, :512]
        out[b] = w @ v
        a = w @ v.abs()
        # a score's error (its sum, the scaling, exp's argument), in nats
        ds = ((x.abs() @ k.abs().T) * scale * SCORE_STEPS * 2 * F32_HALF + s.abs() * 4 * F32_HALF).amax(-1, keepdim=True)
        n = len(ids)
        # exp2 to two units in the last place, sums of n terms in fp32
        dw = ds + 8 * F32_HALF + n * F32_HALF
        otol[b] = out[b].abs() * BF16_HALF + a * (BF16_HALF + 4 * dw) * (1 + 2 * BF16_HALF)
        ltol[b] = (2 * dw + lse[b][:, None].abs() * 8 * F32_HALF).squeeze(-1)
    return out, lse, otol, ltol
