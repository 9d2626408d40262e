"""Embedding gradients of small integers.  Every float32 sum, square and sum of squares is then
exact in any order (below 2^24; the sums of squares above it are float64), so a single position
left out or counted twice changes what is compared, however long the run it is in."""
import numpy as np

# B, T, V, D, tokens.  64: longest samples without block sums for the norms; 256: first batch with
# blocks; 2049: runs past a wave's 64 positions, eight at a time and one left; segments of four waves.
CASES = [
    (1, 1, 3, 8, "one"), (3, 64, 17, 72, "one"), (3, 65, 17, 72, "one"), (1, 255, 5, 7, "one"),
    (1, 256, 5, 7, "one"), (3, 700, 17, 72, "one"), (3, 2049, 17, 72, "one"), (2, 2049, 9, 99, "one"),
    (2, 1000, 6, 520, "two"), (3, 513, 40, 1100, "zipf"), (5, 333, 100, 260, "zipf"),
    (4, 1025, 2, 64, "runs"), (2, 4100, 3, 33, "runs"),
]


def make_case(B, T, V, D, kind, seed=0):
    """(ids [B, T], G [B, T, D] of -3 .. 3 without a zero row, mask or None)."""
    rng = np.random.default_rng([B, T, V, D, seed])
    if kind == "one":
        ids = np.full((B, T), V - 1)
    elif kind == "two":
        ids = np.where(np.arange(T)[None, :] % 3 == 0, 0, V - 1) + np.zeros((B, 1), np.int64)
    elif kind == "runs":       # long runs whose ends fall anywhere among eight positions
        ids = rng.integers(0, V, (B, 1)) + np.zeros((1, T), np.int64)
        ids[:, T // 2 + 3:] = (ids[:, :1] + 1) % V
    else:
        ids = np.minimum((np.exp(rng.random((B, T)) * np.log(V + 1.0)) - 1).astype(np.int64), V - 1)
    G = rng.integers(-3, 4, (B, T, D)).astype(np.float32)
    G[..., 0] = np.where(G[..., 0] == 0, 1, G[..., 0])
    mask = (rng.random((B, T)) < 0.8).astype(np.uint8) if kind in ("zipf", "runs") else None
    return ids.astype(np.int64), G, mask


def exact_sums(ids, G, mask, V):
    """Each sample's gradient [B, V, D] in float64 (integers, exact)."""
    B, T, D = G.shape
    out = np.zeros((B, V, D))
    for i in range(B):
        keep = np.ones(T, bool) if mask is None else mask[i] != 0
        np.add.at(out[i], ids[i][keep], G[i][keep].astype(np.float64))
    return out
