"""Head norms of very small rows, against the float64 oracle.

With elements near s = 2^-64 and eps = 0 the mean square is near 2^-128, a subnormal of spacing
2^-149: each square errs by half of that, their mean and its rounding by 2^-149 in all, 2^-21 of
the mean square and so d = 2^-22 of its root.  That comes to the bounds of ordinary
rows: once for the normalised elements, three times for gradients (r and twice xhat)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from helpers import to_f64
from oracle import attention as A
from test_gpu_attention import DT, E, U, _magnitude, _randn

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -22


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,hq,hkv,D,rot", [(5, 3, 1, 64, 64), (40, 4, 2, 128, 0), (9, 2, 2, 80, 20)])
def test_norm_of_rows_with_a_subnormal_mean_square(T, hq, hkv, D, rot, dtype):
    from activation_sparse_feed_amd import sffn
    rng = np.random.default_rng(T)
    h = sffn.make_heads(T, hq, hkv, D, DT[dtype], rot, 100 if rot else 0, True, 0.0)
    q, k = _randn(rng, (T, hq, D), dtype, 2.0 ** -64), _randn(rng, (T, hkv, D), dtype, 2.0 ** -64)
    w = (1 + _randn(rng, (D,), "f32", 0.3)).to(DT[dtype])
    tab = sffn.rotary_table(100, rot) if rot else None
    pos = torch.from_numpy(rng.integers(0, 100, T).astype(np.int32)).cuda() if rot else None
    gq, gk = _randn(rng, (T, hq, D), dtype), _randn(rng, (T, hkv, D), dtype)
    out = [torch.empty_like(t) for t in (q, k, q, k)]
    gw = [torch.empty(D, device="cuda") for _ in range(2)]
    sffn.qk_norm_rope(h, q, k, w, w, tab, pos, *out[:2])
    sffn.qk_norm_rope_bwd(h, q, k, w, w, tab, pos, gq, gk, *out[2:], *gw, sffn.alloc_heads_workspace(h))
    own = E if dtype == "bf16" else U
    wn, tn, pn = to_f64(w), None if tab is None else to_f64(tab), None if pos is None else pos.cpu().numpy()
    for x, y, g, gx, gwx, heads in ((q, out[0], gq, out[2], gw[0], hq), (k, out[1], gk, out[3], gw[1], hkv)):
        x, g = to_f64(x), to_f64(g)
        want = A.norm_rope(x, wn, tn, pn, rot, False, True, 0.0)
        tol = own * np.abs(want) + ((D + 16) * U + TINY) * _magnitude(x, wn, rot, False, True, 0.0)
        assert (np.abs(to_f64(y) - want) <= tol).all()
        want, want_w = A.norm_rope_backward(x, wn, tn, pn, g, rot, False, True, 0.0)
        pair = _magnitude(g, None, rot, False, False, 0.0)
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True))
        xh = np.abs(x * r)
        scale = r * (pair * np.abs(wn) + xh * (pair * np.abs(wn) * xh).mean(-1, keepdims=True))
        tol = own * np.abs(want) + (2 * (D + 32) * U + 3 * TINY) * scale
        assert (np.abs(to_f64(gx) - want) <= tol).all()
        tol = ((D + 32 + T * heads) * U + TINY) * (pair * xh).sum((0, 1))
        assert (np.abs(to_f64(gwx) - want_w) <= tol).all()
