"""How far partials over an E2M1 cache may be off, row by row.

Only two roundings count: the softmax weights to the queries' type (p (1 + e), |e| <= h,
one e for all of a token's latents) and the output to the partial's type (|e| <= g).  A
row's error is the sum of its tokens' p e c and of g o, so over its 512 columns

    mean square <= h^2 sum_t p_t^2 mean_j c_tj^2 + g^2 mean_j o_j^2 + cross terms,

where the cross terms (two tokens' latents over the columns) have no sign of their own;
SLACK covers them and the fp32 sums and exponentials, each hundreds of times smaller.
The bound is the worst case where one token carries the row, and about 1.7 times the
expected error where many do; a 64-token piece of some thousand tokens left out, or
replaced by its neighbour, is past it in some heads' rows.
"""
import numpy as np

SLACK = 1.25


def parts(q_abs, q_pe, hist, cur, scale, shards, bounds):
    """Per (query token, part): the scores' tokens and softmax weights [H, n] in 64 bits."""
    q = np.concatenate([q_abs, q_pe], -1)
    for i in range(q.shape[0]):
        segs = [hist[lo:hi] for lo, hi in bounds]
        if cur is not None:
            segs.append(cur[:i + 1])
        for p, kv in enumerate(segs):
            if not len(kv):
                yield i, p, kv, None
                continue
            s = scale * (q[i] @ kv.T)
            w = np.exp(s - s.max(1, keepdims=True))
            yield i, p, kv, w / w.sum(1, keepdims=True)


def rms(x):
    return np.sqrt((np.asarray(x, np.float64) ** 2).mean(-1))


def row_bound(w, kv, o, h, g):
    """The bound of the rows' rms errors [H]: weights w [H, n] over tokens kv, outputs o [H, 512]."""
    c2 = (kv[:, :512] ** 2).mean(1)
    return SLACK * np.sqrt(h * h * ((w * w) @ c2) + g * g * (o * o).mean(-1))
