"""Plans for the attention operators: the bucket map of a relative position
bias, made once on the host."""

from __future__ import annotations

import torch


def rel_bucket_map(n_buckets: int, max_distance: int, two_sided: bool,
                   device=None) -> torch.Tensor:
    """Bucket of each distance -max_distance ... max_distance (key position
    minus query position), int32, as the bias calls take it: they take maps of
    max_distance up to 1024.

    Two-sided, the upper half of the buckets serves the keys after the query;
    one-sided, those share bucket 0 with the query's own position.  On a side
    with n buckets the first e = max(1, n // 2) distances have one each, and a
    distance a >= e has bucket

        e + floor((n - e) log(a / e) / log(max_distance / e)),  at most n - 1.

    Buckets are decided by comparing whole powers, a^(n-e) against
    e^(n-e-k) max_distance^k, so a distance that lies on a border (16, 32, ...
    with 8 and 128) is never moved by a rounded logarithm."""
    n = n_buckets // 2 if two_sided else n_buckets
    if n < 1:
        raise ValueError("each side needs a bucket")
    e = max(1, n // 2)
    if max_distance < 1 or (n > 1 and max_distance <= e):
        raise ValueError(f"max_distance must be larger than the {e} distances with buckets of "
                         "their own")
    # first distance of bucket e + k, k = 1 ... n - e - 1
    borders = []
    a = e
    for k in range(1, n - e):
        while a ** (n - e) < e ** (n - e - k) * max_distance ** k:
            a += 1
        borders.append(a)
    side = []
    for a in range(max_distance + 1):
        side.append(min(a, n - 1) if a < e or n == 1 else e + sum(a >= b for b in borders))
    if two_sided:
        out = side[:0:-1] + [side[0]] + [n + b for b in side[1:]]
    else:
        out = side[:0:-1] + [side[0]] + [side[0]] * max_distance
    return torch.tensor(out, dtype=torch.int32, device=device)
