"""gdn_rope and gdn_rope_bwd against the fp64 definition, against differences,
and on the layouts, widths and positions that a caller may have."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention_ref as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows(B, H, T, d, dt, layout, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, H, T, d, generator=g, device="cuda").to(dt)
    if layout == "bthd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "wide":      # rows inside longer ones, as a fused projection leaves them
        w = torch.full((B, T, H, d + 32), float("nan"), dtype=dt, device="cuda")
        w[..., 16:16 + d] = x.transpose(1, 2)
        return w[..., 16:16 + d].transpose(1, 2)
    return x


def bound(x, half, adjacent, y, dt):
    """Two products and a sum, each rounded to fp32 (2^-24 each of the products' magnitudes,
    where |cos|, |sin| <= 1), then one rounding to dt; doubled."""
    a = np.abs(x[..., 0:2 * half:2] if adjacent else x[..., :half])
    b = np.abs(x[..., 1:2 * half:2] if adjacent else x[..., half:2 * half])
    e = np.zeros_like(x)
    both = 2 * (a + b) * 2.0 ** -24
    if adjacent:
        e[..., 0:2 * half:2] = e[..., 1:2 * half:2] = both
    else:
        e[..., :half] = e[..., half:2 * half] = both
    return 2 * (e + (np.abs(y) * 2.0 ** -9 if dt == torch.bfloat16 else 0))


CASES = [
    # B, Hq, Hk, T, d, rot, axes, adjacent, layout, io
    (2, 4, 2, 37, 128, 128, 1, False, "bhtd", "bf16"),
    (1, 3, 1, 1, 64, 64, 1, False, "bthd", "bf16"),
    (3, 5, 5, 65, 64, 32, 3, False, "bthd", "f32"),
    (2, 2, 1, 33, 256, 256, 3, True, "wide", "bf16"),
    (1, 7, 2, 129, 128, 64, 2, True, "bhtd", "f32"),
    (2, 3, 1, 19, 80, 48, 4, False, "wide", "f32"),
    (1, 1, 1, 300, 48, 16, 1, True, "bthd", "bf16"),
    (2, 2, 2, 9, 16, 16, 2, False, "bhtd", "f32"),
    (1, 2, 1, 5, 64, 0, 1, False, "bhtd", "bf16"),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,T,d,rot,axes,adjacent,layout,io", CASES)
def test_matches_definition(B, Hq, Hk, T, d, rot, axes, adjacent, layout, io, back):
    dt = DT[io]
    q, k = rows(B, Hq, T, d, dt, layout, 1), rows(B, Hk, T, d, dt, layout, 2)
    rng = np.random.default_rng(d + T)
    pos = rng.integers(0, 1000, (axes, B, T)).astype(np.int32)
    which = [i % axes for i in range(rot // 2)]
    cos, sin = gdn.gdn_rope_table(1000, rot)
    f = gdn.gdn_rope_bwd if back else gdn.gdn_rope
    yq, yk = f(q, k, cos, sin, torch.from_numpy(pos).cuda(), axes=which, adjacent=adjacent,
               check=True)
    for x, y in ((q, yq), (k, yk)):
        ref = np.stack([R.rotate(U.f64(x[b]), U.f64(cos), U.f64(sin), pos[:, b], which, adjacent,
                                 back) for b in range(B)])
        assert y.dtype == dt and y.shape == x.shape
        assert np.all(np.abs(U.f64(y) - ref) <= bound(U.f64(x), rot // 2, adjacent, ref, dt))


def test_no_keys_shared_positions_and_in_place():
    q = rows(2, 3, 50, 64, torch.float32, "bhtd", 3)
    cos, sin = gdn.gdn_rope_table(64, 64)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    y, none = gdn.gdn_rope(q, None, cos, sin, pos, check=True)
    assert none is None
    y2, _ = gdn.gdn_rope(q, None, cos, sin, pos[None].expand(2, -1).contiguous(), check=True)
    assert torch.equal(y, y2)
    z = q.clone()
    gdn.gdn_rope(z, None, cos, sin, pos, out=(z, None), check=True)
    assert torch.equal(y, z)


def test_gradient_is_the_transpose():
    # L = <w, R x>: dL/dx by gdn_rope_bwd; R is linear, so a central difference of any step is
    # exact but for rounding: 2^-24 of each of the sums' terms, some 4 roundings each
    q, k = rows(2, 3, 21, 64, torch.float32, "bthd", 4), rows(2, 1, 21, 64, torch.float32, "bthd", 5)
    wq, wk = rows(2, 3, 21, 64, torch.float32, "bhtd", 6), rows(2, 1, 21, 64, torch.float32, "bhtd", 7)
    uq, uk = rows(2, 3, 21, 64, torch.float32, "bthd", 8), rows(2, 1, 21, 64, torch.float32, "bthd", 9)
    cos, sin = gdn.gdn_rope_table(40, 48)
    which = gdn.gdn_rope_axes((8, 8, 8), interleave=True)
    pos = torch.randint(0, 40, (3, 2, 21), dtype=torch.int32, device="cuda")
    kw = dict(axes=which, check=True)
    gq, gk = gdn.gdn_rope_bwd(wq, wk, cos, sin, pos, **kw)

    def loss(e):
        a, b = gdn.gdn_rope(q + e * uq, k + e * uk, cos, sin, pos, **kw)
        return (wq.double() * a.double()).sum() + (wk.double() * b.double()).sum()

    diff = (loss(1.0) - loss(-1.0)) / 2
    grad = (gq.double() * uq.double()).sum() + (gk.double() * uk.double()).sum()
    size = (wq.double() * (q.double().abs() + uq.double().abs())).abs().sum() * 2
    assert abs(float(diff - grad)) <= float(size) * 2.0 ** -20
    # and there and back is the identity
    a, b = gdn.gdn_rope(q, k, cos, sin, pos, **kw)
    a, b = gdn.gdn_rope_bwd(a, b, cos, sin, pos, **kw)
    assert float((a - q).abs().max()) <= float(q.abs().max()) * 2.0 ** -20
    assert float((b - k).abs().max()) <= float(k.abs().max()) * 2.0 ** -20


def test_empty_and_nonfinite_rows():
    cos, sin = gdn.gdn_rope_table(8, 64)
    e = torch.empty(2, 3, 0, 64, device="cuda")
    y, _ = gdn.gdn_rope(e, None, cos, sin, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert y.shape == e.shape
    q = rows(1, 2, 4, 64, torch.float32, "bhtd", 10)
    clean, _ = gdn.gdn_rope(q, None, cos, sin, torch.arange(4, dtype=torch.int32, device="cuda"))
    q[0, 1, 2, 5] = float("nan")
    y, _ = gdn.gdn_rope(q, None, cos, sin, torch.arange(4, dtype=torch.int32, device="cuda"))
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[0, 1, 2, 5] = bad[0, 1, 2, 37] = True
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("bad", [-1, 8])
def test_position_outside_the_table_is_reported(bad):
    cos, sin = gdn.gdn_rope_table(8, 64)
    q = rows(1, 2, 4, 64, torch.float32, "bhtd", 11)
    pos = torch.tensor([0, 1, bad, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_rope(q, None, cos, sin, pos, check=True)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    gdn.sync_check()      # reported once


def test_on_another_stream():
    q = rows(2, 4, 512, 128, torch.bfloat16, "bhtd", 12)
    cos, sin = gdn.gdn_rope_table(512, 128)
    pos = torch.arange(512, dtype=torch.int32, device="cuda")
    want, _ = gdn.gdn_rope(q, None, cos, sin, pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.zeros_like(q)
        for _ in range(20):
            x.add_(0)
        x.copy_(q)                                  # the call has to wait for this
        got, _ = gdn.gdn_rope(x, None, cos, sin, pos)
    side.synchronize()
    assert torch.equal(want, got)
