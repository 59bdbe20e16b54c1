"""The selective scan over more sequences than a grid's second axis takes: pixels of a map as the batch.
Tolerances as in test_gpu_mixer.py."""
import numpy as np
import pytest
import torch

import mixer_ref as M
from test_gpu_mixer import Out, near, scan_data, space

pytestmark = pytest.mark.gpu

B0, TIMES = 100, 700  # distinct sequences, and how often each is there: 70000


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


@pytest.mark.parametrize("L,D,N", [(3, 4, 4), (19, 5, 7)])
def test_seventy_thousand_sequences(hc, L, D, N):
    t, B = torch.float32, B0 * TIMES
    x, r = scan_data(B0, L, D, 1, N, t, True, True, None, 0, seed=50)
    lens = [(L, 0, 1, L - 1)[i % 4] for i in range(B0)]
    ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], 1, True, r["D"], r["z"], r["bias"], r["h0"], lens, r["gy"],
                 r["ghT"])
    many = {k: x[k].repeat(TIMES, 1, 1) for k in ("u", "dt", "Bm", "Cm", "z", "gy", "h0", "ghT")}
    d = hc.selective_scan_desc(B, L, D, N, t)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 1))
    saved = space(hc, hc.hc_selective_scan_saved_size(d))[0]
    kw = dict(D=x["D"], z=many["z"], dt_bias=x["bias"], h0=many["h0"], ws=ws, ws_bytes=nb,
              lens=torch.tensor(lens * TIMES, dtype=torch.int32, device="cuda"))
    args = (many["u"], many["dt"], x["A"], many["Bm"], many["Cm"])
    y, hT = Out((B, L, D)), Out((B, D, N))
    hc.check(hc.hc_selective_scan_fwd(d, *args, y.t, hT=hT.t, saved=saved, **kw))
    o = dict(gu=Out((B, L, D)), gdt=Out((B, L, D)), gA=Out((D, N)), gB=Out((B, L, N)), gC=Out((B, L, N)))
    rest = dict(gz=Out((B, L, D)), gD=Out((D,)), gdt_bias=Out((D,)), gh0=Out((B, D, N)))
    hc.check(hc.hc_selective_scan_bwd(d, *args, many["gy"], saved, *(v.t for v in o.values()), ghT=many["ghT"],
                                      **{k: v.t for k, v in rest.items()}, **kw))
    for k, v in dict(o, y=y, state=hT, gstate=rest.pop("gh0"), **rest).items():
        if k in ("gA", "gD", "gdt_bias"):
            near(k, v, ref[k] * TIMES, 1e-4)
        else:
            near(k, v, np.tile(ref[k], (TIMES, 1, 1)), 1e-5)


def test_one_token_of_seventy_thousand_sequences(hc):
    t, B, D, N = torch.float32, B0 * TIMES, 12, 16
    x, r = scan_data(B0, 1, D, 1, N, t, True, True, None, 0, seed=51)
    ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], 1, True, r["D"], r["z"], r["bias"], r["h0"])
    row = {k: x[k][:, 0].repeat(TIMES, 1) for k in ("u", "dt", "Bm", "Cm", "z")}
    state, y = Out((B, D, N)), Out((B, D))
    state.t.copy_(x["h0"].repeat(TIMES, 1, 1))
    hc.check(hc.hc_selective_scan_step(hc.selective_scan_desc(B, 1, D, N, t), row["u"], row["dt"], x["A"], row["Bm"],
                                       row["Cm"], state.t, y.t, D=x["D"], z=row["z"], dt_bias=x["bias"]))
    near("y", y, np.tile(ref["y"][:, 0], (TIMES, 1)), 1e-5)
    near("state", state, np.tile(ref["state"], (TIMES, 1, 1)), 1e-5)
