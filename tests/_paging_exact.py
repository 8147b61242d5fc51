"""Attention over pages in 64 bits with tolerances that stay small on long sequences.

A value is o = sum_j w_j v_j.  Its error, from the arithmetic:
 - a weight is rounded to fp16 before the product with V, half a step: 2^-11 of it, or,
   where it is subnormal there, 2^-25 of the reference that it stands against.  The
   reference lies at least 2^7 below the largest weight of the keys that share it, so the
   latter is 2^-32 of that weight, for weights below 2^-21 of it only;
 - its exponent is an fp32 score (products and sums of at most 128 terms, span = sum |q k|
   scale) and the exponential's own 2^-22: 2 span 2^-22;
 - O is summed by MMAs of 16 keys.  At most 2048 keys, 128 MMAs, go into one sum before
   it is added to that of the keys before; an MMA's 17 terms are cut off at 2^-24 of the
   largest at worst: 128 * 17 * 2^-24, and as much again for the sum of the weights and for
   what the pieces lose when they are joined: 2^-12 in all;
 - the result is rounded to fp16: 2^-11 of it, or 2^-25."""
import torch

import _paging_ref as pref


def tolerance(w, v, want, span, rounded=True):
    """w [H, n] normalised weights, v [H, n, D], want [H, D], span [H]: tolerance [H, D].
    rounded: whether rounding to fp16 changes a weight."""
    part = 2.0 ** -12 + 2 * span * 2.0 ** -22 + (2.0 ** -11 if rounded else 0.0)
    tol = part[:, None] * torch.einsum("hj,hjd->hd", w, v.abs())
    top = w.amax(-1)
    tiny = (w < 2.0 ** -21 * top[:, None]).to(w.dtype)
    tol += 2.0 ** -32 * top[:, None] * torch.einsum("hj,hjd->hd", tiny, v.abs())
    return tol + 2.0 ** -11 * want.abs() + 2.0 ** -25


def sequence(q, kc, vc, codec, entries, n, scale, rounded=True):
    """(want, tol) [H, D] of one sequence, q [H, D], all of whose n rows are there."""
    g = q.shape[0] // kc.shape[1]
    want, tol = [], []
    for hk in range(kc.shape[1]):
        k = pref.gather(kc[:, hk:hk + 1], entries, n, codec)[0][0]
        v = pref.gather(vc[:, hk:hk + 1], entries, n, codec)[0][0]
        x = q[hk * g:(hk + 1) * g].double()
        w = torch.softmax(x @ k.T * scale, -1)
        span = (x.abs() @ k.abs().T * abs(scale)).amax(-1)
        o = w @ v
        want.append(o)
        tol.append(tolerance(w, v.expand(g, *v.shape), o, span, rounded))
    return torch.cat(want), torch.cat(tol)


def striped(pages, page, d, seg, dtype=torch.float32):
    """Rows [pages, 1, page, d] of ones and zeros: row j of page i has a one at dim (j' // seg)
    % d, j' = i page + j, so that each dim of their mean counts the keys of its stripes."""
    at = torch.arange(pages * page) // seg % d
    return torch.nn.functional.one_hot(at, d).to(dtype).view(pages, 1, page, d)
