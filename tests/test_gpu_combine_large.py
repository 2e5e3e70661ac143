"""The sum of a token's experts and its gradients where the rows are too many for the
caches, in whole and ragged lengths, on tokens picked out of all."""
import numpy as np
import pytest

import precision_integer_gemm_amd as L
import routing_reference as R
from test_gpu_routing import HALF_STEP, LEAST, kind_of, torch  # noqa: F401

pytestmark = pytest.mark.gpu


# rows of 108, 213, 117 and 219 MB, of up to 2048 values and of more
@pytest.mark.parametrize("kind,T,top,N", [("float32", 6600, 2, 2045), ("float32", 13000, 2, 2048), ("bfloat16", 3500, 4, 4173), ("float16", 5500, 5, 3990)])
def test_rows_past_the_caches(torch, kind, T, top, N):  # noqa: F811
    g = torch.Generator("cuda").manual_seed(T)
    dtype = kind_of(torch, kind)
    rows = T * top + 5
    y = torch.randn(rows, N, device="cuda", generator=g).to(dtype)
    dout, residual = (torch.randn(T, N, device="cuda", generator=g).to(dtype) for _ in range(2))
    places = torch.randperm(rows, device="cuda", generator=g)[:T * top].int().view(T, top).clone()
    places[::7, 1] = -1
    w = torch.randn(T, top, device="cuda", generator=g)
    out = L.lpgemm_combine(y, places, w, residual=residual)
    dy, dw = L.lpgemm_combine_backward(dout, y, places, w, dy=torch.full_like(y, 3.0))
    some = np.array([0, 1, 7, T // 2, T - 2, T - 1])
    p, wv = places.cpu().numpy()[some], w.cpu().numpy()[some]
    used = np.zeros(rows, bool)
    used[places.cpu().numpy()[places.cpu().numpy() >= 0]] = True
    assert (dy[torch.from_numpy(~used).cuda()] == 3).all()
    for t, at, weight in zip(some, p, wv):
        rowsof = [int(a) for a in at if a >= 0]
        yv = y[rowsof].double().cpu().numpy()
        want, size = R.combine(yv, np.array([[rowsof.index(a) if a >= 0 else -1 for a in at]], np.int32), weight[None], residual[t:t + 1].double().cpu().numpy())
        step = 1.01 * (top + 1) * 2.0 ** -24 * size
        off = np.abs(out[t:t + 1].double().cpu().numpy() - want)
        assert (off <= step + HALF_STEP[kind] * (np.abs(want) + step) + LEAST[kind]).all()
        d = dout[t].double().cpu().numpy()
        for k, a in enumerate(at):
            if a < 0:
                assert dw[t, k] == 0
                continue
            v = float(weight[k]) * d
            assert (np.abs(dy[int(a)].double().cpu().numpy() - v) <= (2.0 ** -24 + HALF_STEP[kind]) * 1.001 * np.abs(v) + LEAST[kind]).all()
            terms = d * yv[rowsof.index(a)]
            steps = -(-N // 2048) * 8 + 6 + 3  # of a lane and column, 8 columns, 64 lanes, 4 waves
            assert abs(float(dw[t, k]) - terms.sum()) <= 1.01 * steps * 2.0 ** -24 * np.abs(terms).sum()
