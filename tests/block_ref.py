"""Plain 64-bit forms of the 8-bit and mixture-of-experts operators, on the
CPU, for their GPU tests.  Not collected by pytest."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half the smallest step


def dtype(name):
    import torch

    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
            "e4m3": torch.float8_e4m3fn}[name]


def padded(t, unit, extra=0, fill=float("nan")):
    """`t` (CPU) on the GPU as a view whose rows lie in a wider buffer filled
    with `fill`, strides a multiple of `unit`."""
    import torch

    *lead, n = t.shape
    ld = max(unit, -(-n // unit) * unit) + extra * unit
    wide = torch.full((*lead, ld), fill, dtype=torch.float32).to(t.dtype)
    wide[..., :n] = t
    return wide.cuda()[..., :n]


def block_product(A, SA, B, SB):
    """(C, bound on the fp32 error) in 64 bits.  A (M x K), B (N x K): arrays
    of values; SA (kb x M), SB (nb x kb), or None for plain products."""
    A, B = A.astype(np.float64), B.astype(np.float64)
    K = A.shape[1]
    kb = -(-K // 128)
    if SA is not None:
        A = A * np.repeat(SA.astype(np.float64).T, 128, 1)[:, :K]
        B = B * np.repeat(np.repeat(SB.astype(np.float64), 128, 0)[:B.shape[0]], 128, 1)[:, :K]
    C, mag = A @ B.T, np.abs(A) @ np.abs(B).T
    # each product passes at most 128 sums of its block (of K for 16-bit
    # types) and kb sums of blocks and of wave parts, each at most one fp32
    # step (2 U) off, and two roundings of the scales
    sums = (128 if SA is not None else K) + kb + 16
    return C, 2 * U * sums * mag


def cut_bound(A, SA, B, SB):
    """What a 16-bit C of e4m3 operands may miss beside its fp32 error: of
    eight products at a time all but the largest are cut by less than 2^-13 of
    its codes' powers of two (2^-6 for subnormal codes), times the scales."""
    def power(x):
        x = np.maximum(np.abs(x.astype(np.float64)), 2.0 ** -6)
        x = np.pad(x, ((0, 0), (0, -x.shape[1] % 128)), constant_values=2.0 ** -6)
        return 2.0 ** np.floor(np.log2(x)).reshape(len(x), -1, 8)

    pa, pb = power(A), power(B)
    cut = np.zeros((len(pa), len(pb)))
    for i in range(pa.shape[1]):  # eights; 16 to a block
        largest = (pa[:, i][:, None] * pb[:, i][None]).max(2)
        scale = np.abs(SA[i // 16][:, None] * np.repeat(SB[:, i // 16], 128)[:len(pb)][None])
        cut += 7 * 2.0 ** -13 * largest * scale
    return cut


def check_rounded(got, want, err, out):
    """got (float64) is `want`, known to `err`, rounded once to type `out`."""
    tol = err + HALF_STEP[out] * (np.abs(want) + err) + TINY[out]
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(off / tol)), np.argwhere(bad)[:4].tolist())


def plan(ids, E):
    """(offsets, rows, pos) of ids (T x k); ids outside 0 .. E-1 are dropped."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    rows = np.full(flat.size, -1)
    pos = np.full(flat.size, -1)
    n = offsets[E]
    rows[:n] = order[:n] // ids.shape[1]
    pos[order[:n]] = np.arange(n)
    return offsets, rows, pos.reshape(ids.shape)


def route(x, k, bias=None, score="softmax", groups=1, topk_groups=None, group_top=2,
          renormalize=True, scale=1.0):
    """(ids, weights) in 64 bits; the order without a bias is that of the
    logits.  Equal scores go by logit (groups by that of their best expert),
    then by index."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    x = np.minimum(x, float(np.finfo(np.float32).max))
    T, E = x.shape
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = x.max(1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            e = np.exp(x - m)
            z = e.sum(1, keepdims=True)
            s = e / np.where(z > 0, z, 1.0)
        else:
            s = 1 / (1 + np.exp(-x))
    c = s if bias is None else s + bias.astype(np.float64)
    if bias is None and (groups == 1 or group_top == 1):
        c = x
    c = np.where(np.isneginf(x), -np.inf, c)  # masked, whatever the bias
    topk_groups = groups if topk_groups is None else topk_groups
    ids = np.zeros((T, k), np.int64)
    size = E // groups
    for t in range(T):
        by = c[t].reshape(groups, size)
        top = -np.sort(-by, 1)[:, :group_top]
        best = np.where(np.isneginf(top[:, 0]), -np.inf, np.where(np.isneginf(top), 0, top).sum(1))
        order = np.lexsort((np.arange(E), -x[t], -c[t]))  # by c, then logit, then index
        first = [x[t][order[order // size == b][0]] for b in range(groups)]
        kept = np.lexsort((np.arange(groups), -np.array(first), -best))[:topk_groups]
        ids[t] = order[np.isin(order // size, kept)][:k]
    w = np.take_along_axis(s, ids, 1)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return ids, w * scale
