"""What the row operators' tests of single terms share: how many additions lie
between a term and its sum in the kernels, and inputs in which one term at a
border of the kernels' work (a vector, a round, a tile, a workgroup) decides
the result, so that a term lost or counted twice there cannot hide in a
tolerance."""
import numpy as np

from oracle import rows


# ------------------------------------------------------------------ depths
def norm_depth(N):
    """A thread's elements one after the other (at most 8 NV), 6 levels in the
    wave and one for each doubling of a row's waves; the forward has the most."""
    for width, most in ((512, 8 + 6), (1024, 16 + 6), (2048, 16 + 6 + 1), (4096, 16 + 6 + 2),
                        (8192, 32 + 6 + 2)):
        if N <= width:
            return most
    return 32 + 6 + 3


def norm_groups(N):
    """Rows that a workgroup of the backward holds at once."""
    return 16 if N <= 512 else 8 if N <= 1024 else 4 if N <= 2048 else 2 if N <= 4096 else 1


def norm_rows_depth(M, N):
    """A group's rows one after the other, the groups of a workgroup, then
    sixteen ranges of at most sixteen workgroups."""
    g = norm_groups(N)
    return -(-M // (256 * g)) + g + 16 + 16


def distill_depth(V):
    """A round of 32 logits a lane is 12 additions (a vector's, then the
    vectors') and a factor on each side of the join with the sum so far, 4
    together; a row is at most 8 rounds, or pieces of at most 4. Then the lanes
    (a factor, 6 levels: 10) and the four waves (3 joins of 4), and with pieces
    a lane's parts and the lanes again."""
    n = -(-(V + 63) // 8192)
    p = 1 if n <= 8 else -(-n // 4)
    h = 16 * -(-n // p) + 10 + 12
    return h if p == 1 else h + 4 * -(-4 * p // 64) + 10


def embed_depth(M, count):
    """A tile's tokens, then the tiles' parts in eight ranges, and the ranges."""
    tile = 32 if M <= 32 or M > 4096 else 16
    return tile + -(-(-(-count // tile) + 1) // 8) + 8 + 1


# ------------------------------------------------------------------- inputs
def norm_places(N):
    """The row's ends (whole, as a vector may be moved back by one to eight
    elements) and both sides of every width that threads and vectors cover."""
    at = {0, 1, 7, 8} | set(range(N - 10, N))
    for w in (256, 512, 1024, 2048, 4096, 8192):
        at |= {w - 1, w}
    return sorted(p for p in at if 0 <= p < N)


def norm_case(N, seed):
    """One row for each place: x and dY there are sqrt(N) / 2, so that the place
    is a fifth of the row's squares and of the sums of the backward."""
    g = np.random.default_rng(seed)
    at = norm_places(N)
    x, dY = g.standard_normal((len(at), N)), g.standard_normal((len(at), N))
    big = max(3.0, 0.5 * np.sqrt(N))
    x[np.arange(len(at)), at] = big
    dY[np.arange(len(at)), at] = big
    return x.astype(np.float32), dY.astype(np.float32), at


def distill_places(V):
    if V <= 300:
        return list(range(V))
    at = {0, 1, 7, 8, V - 9, V - 8, V - 2, V - 1}
    n = -(-(V + 63) // 8192)
    p = 1 if n <= 8 else -(-n // 4)
    step = -(-n // p)
    for k in {1, 2, step - 1, step, step + 1, 2 * step, n - 1}:
        # a row's rounds begin with the line of 64 or 32 logits in which it begins
        at |= {8192 * k + o for o in (-65, -64, -63, -33, -32, -31, -9, -8, -1, 0, 1)}
    return sorted(v for v in at if 0 <= v < V)


def distill_case(V, T, seed):
    """One row for each place: its logit there is as much as all others
    together, and the teacher names it and its neighbours, once again elsewhere."""
    g = np.random.default_rng(seed)
    at = np.array(distill_places(V))
    M = at.size
    z = (2.5 * g.standard_normal((M, V))).astype(np.float32)
    r = np.arange(M)
    z[r, at] = -np.inf
    z[r, at] = T * np.log(np.exp(z.astype(np.float64) / T).sum(1)) if V > 1 else 1.0
    ids = np.stack([at, np.minimum(at + 1, V - 1), np.maximum(at - 1, 0), at,
                    g.integers(0, V, M), g.integers(0, V, M)], 1)
    t = g.standard_normal((M, 6)).astype(np.float32)
    return z, ids, t, at


def embed_places(M):
    at = {0, 1, 2, M - 3, M - 2, M - 1}
    for w in (8, 16, 32, 64, 128, 256, 512, 1024, 2048, 4096, 8192):
        at |= {w - 1, w, w + 1, M // w * w - 1, M // w * w}
    return sorted(p for p in at if 0 <= p < M)


def embed_case(M, seed):
    """All tokens share one id; column j has a large value at the j-th place."""
    g = np.random.default_rng(seed)
    at = embed_places(M)
    dY = g.standard_normal((M, len(at)))
    dY[at, np.arange(len(at))] = 500.0
    return dY.astype(np.float32), at


def rows_case(M, N, seed):
    """dY of which column j has a large value in one row at a border of the
    workgroups' shares (dgamma and dbeta are sums over the rows)."""
    g = np.random.default_rng(seed)
    b = norm_groups(N)
    at = sorted({p for w in (1, b, 16 * b, 128 * b, 255 * b, 256 * b) for p in (w - 1, w, M - w)
                 if 0 <= p < M})
    dY = g.standard_normal((M, N))
    x = g.standard_normal((M, N))
    for j in range(min(N, 4 * len(at))):
        dY[at[j % len(at)], j] = 500.0
        x[at[j % len(at)], j] = 2.0
    return x.astype(np.float32), dY.astype(np.float32), at


def tolerance(want, err, eps):
    """What a GPU result may be off by: err, half a step of its type, half of
    the smallest subnormal."""
    return err + 0.5 * eps * (np.abs(want) + err) + 2.0 ** -126 * eps


__all__ = [n for n in dir() if n.endswith(("_case", "_depth", "_places", "_groups"))] + ["tolerance", "rows"]
