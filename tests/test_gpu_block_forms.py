"""Forms of linear attention and of the norms around a block that one call
takes alone: a single norm over many rows of a workgroup, and what else the
sizes of the other files do not reach.

Tolerances as in test_gpu_block_ops.py where nothing else is derived.
"""
import numpy as np
import pytest

import oracle.block_oracle as L
from tests.test_gpu_layer_ops import check, dev_of, round_to

pytestmark = pytest.mark.gpu


def ops():
    from gated_delta_rule_recurrence_amd import ops
    return ops


# ---- the norms: one of them, several rows a workgroup ------------------------------

# rows a workgroup of 256, 512 and 1024 lanes takes several of, in either direction
ROWS = ((3000, 600), (1100, 2304), (700, 4104))


def norm_rows(dtype, rows, C, post, pre, center, gate, seed):
    """Rows of very different sizes (2^-6 to 2^6), so that the statistics of
    one show in another's."""
    r = np.random.default_rng(seed)
    size = 2.0 ** r.integers(-6, 7, size=(rows, 1))
    n = lambda: round_to(r.normal(size=(rows, C)) * size, dtype)
    d = dict(x=n(), res=n(), dy=round_to(r.normal(size=(rows, C)), dtype), dh=round_to(r.normal(size=(rows, C)), dtype))
    d["gate"] = round_to(r.normal(size=(rows if gate == "row" else 1, C)), dtype) if gate else None
    w = [round_to(1 + 0.2 * r.normal(size=C), dtype) if use else None for use in (post, pre)]
    b = [round_to(r.normal(size=C), dtype) if center and use else None for use in (post, pre)]
    d["w"] = (w[0], b[0], w[1], b[1])
    return d


@pytest.mark.parametrize("dtype,gate", (("bf16", "row"), ("f32", "channel")))
@pytest.mark.parametrize("post,pre,center", ((0, 1, 0), (1, 0, 0), (0, 1, 1), (1, 0, 1)))
@pytest.mark.parametrize("rows,C", ROWS + ((3100, 1001),))
def test_res_one_norm_many_rows(cuda, rows, C, post, pre, center, dtype, gate):
    import torch
    d = norm_rows(dtype, rows, C, post, pre, center, gate, seed=C + post)
    on = lambda a: dev_of(a, dtype, cuda)
    g = None if d["gate"] is None else on(d["gate"]) if gate == "row" else on(d["gate"])[0]
    args = [on(d["x"]), on(d["res"]), g, *map(on, d["w"])]
    how = dict(alpha=0.6, eps=1e-5, post=bool(post), pre=bool(pre), center=bool(center))
    y, h, stats = ops().gdr_res_forward(*args, **how)
    back = lambda: ops().gdr_res_backward(*args, stats, on(d["dy"]) if pre else None, on(d["dh"]), **how)
    grads = back()
    for _ in range(3):
        again = ops().gdr_res_forward(*args, **how)
        for a, b in zip((y, h, stats, *grads), (*again, *back())):
            assert a is None and b is None or torch.equal(a, b)
    host = (d["x"], d["res"], d["gate"], *d["w"], 0.6, 1e-5, post, pre, center)
    ref, mag = (L.res_forward(*host, mag=m) for m in (False, True))
    if pre:
        check("y", y, ref[0], mag[0], dtype, 128)
    check("h", h, ref[1], mag[1], dtype, 128)
    ref, mag = (L.res_backward(*host, dy=d["dy"], dh=d["dh"], mag=m) for m in (False, True))
    given = (1, 1, g, *d["w"])
    for i, name in enumerate(("dx", "dr", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b")):
        if given[i] is None:
            assert grads[i] is None
        else:
            check(name, grads[i], ref[i], mag[i], dtype, 256 + (rows if i >= 2 else 0))


@pytest.mark.parametrize("post,pre,center", ((1, 1, 0), (0, 1, 0), (1, 0, 1)))
@pytest.mark.parametrize("rows,C", ROWS)
def test_res_in_place_many_rows(cuda, rows, C, post, pre, center):
    """h over the residual and y over x, with the next row in flight."""
    import torch
    x, r = (torch.randn(rows, C, device=cuda).bfloat16() for _ in range(2))
    w = torch.rand(C, device=cuda).bfloat16()
    args = (None, w if post else None, None, w if pre else None)
    how = dict(post=bool(post), pre=bool(pre), center=bool(center), save=False)
    y, h, _ = ops().gdr_res_forward(x, r, *args, **how)
    a, b, _ = ops().gdr_res_forward(x, r, *args, **how, y=x if pre else None, h=r)
    assert b is r and torch.equal(r, h) and (not pre or a is x and torch.equal(x, y))
