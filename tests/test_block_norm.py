"""GPU: the norms around a block through the C ABI, against their definition in 64 bits and its
automatic differentiation.

Tolerances (layer_reference.close): half a step of a 16-bit output, and fp32 roundings counted as for
layer norm: 128 for a norm (sums added in fewer than 64 steps, root and quotient), here two of them and the gate
(an exponential and a quotient, 16 units with its argument): 300; a gradient over the rows adds one per row.  They count in
units of the largest value times how far a row's values exceed their deviation, which the subtraction
of the mean and the reciprocal deviation scale errors by."""
import pytest
import torch

import layer_reference as ref
from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]
DEV = "cuda"
NAMES = ("x", "residual", "z", "scale", "post_weight", "post_bias", "weight", "bias")


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def inputs(types, rows, D, gate=True, scale=True, weights=True, biases=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt, rt = types
    t = dict(x=normal(g, rows, D, dtype=dt), residual=normal(g, rows, D, dtype=rt, scale=2.0),
             z=normal(g, rows, D, dtype=dt) if gate else None, scale=normal(g, D, scale=0.5) if scale else None)
    for name in ("post_weight", "post_bias", "weight", "bias"):
        given = biases if name.endswith("bias") else weights
        t[name] = (normal(g, D, scale=0.2) + (0 if name.endswith("bias") else 1)) if given else None
    return t, dict(dy=normal(g, rows, D, dtype=dt), dresidual_out=normal(g, rows, D, dtype=rt))


def norm64(x, w, b, eps, rms):
    return ref.norm(dict(x=x, weight=w, bias=b), eps, rms)


def block64(u, eps, rms, post):
    zero = dict(weight=u["post_weight"], bias=u["post_bias"])
    if post:
        p = norm64(u["x"], u["post_weight"], u["post_bias"], eps, rms)
    else:
        p = u["x"] if zero["weight"] is None else u["x"] * zero["weight"]
        p = p if zero["bias"] is None else p + zero["bias"]
    if u["z"] is not None:
        p = p / (1 + torch.exp(-u["z"]))
    if u["scale"] is not None:
        p = p * u["scale"]
    h = u["residual"] + p
    return norm64(h, u["weight"], u["bias"], eps, rms), h


def ratio_of(x, eps, rms):
    """How far a row's values exceed their deviation."""
    if not x.numel():
        return 1.0
    dev = torch.sqrt(((x if rms else x - x.mean(-1, keepdim=True)) ** 2).mean(-1) + eps)
    return max(1.0, float((x.abs().amax(-1) / dev).max())), dev


def args(t):
    return [t[k] for k in NAMES]


def check(lib, t, grads, rms, post, label, eps=1e-5, dres=True):
    kind = dict(eps=eps, rms=rms, post=post)
    y, h = lib.block_norm_fwd(*args(t), **kind)
    u = ref.in_64_bits(t, grad=True)
    y64, h64 = block64(u, eps, rms, post)
    r1, dev1 = ratio_of(u["x"].detach(), eps, rms)
    r2, dev2 = ratio_of(h64.detach(), eps, rms)
    branch = float((h64 - u["residual"]).detach().abs().max()) if t["x"].numel() else 0.0
    top = float(h64.detach().abs().max()) if t["x"].numel() else 1.0
    first = r1 if post else 1.0
    ref.close(h, h64, 150 * first, label + " h", scale=max(top, branch))
    # an error of h is one of y by the reciprocal deviation
    through = max(1.0, float((top / dev2).max()))
    ref.close(y, y64, 300 * first * r2, label + " y", scale=max(float(y64.detach().abs().max()), through))
    out = lib.block_norm_bwd(*args(t), **kind, dy=grads["dy"], dresidual_out=grads["dresidual_out"] if dres else None)
    want = ref.gradients([y64, h64], [grads["dy"], grads["dresidual_out"] if dres else None], u)
    rows = t["x"].shape[0]
    # dh is a difference of terms of the size of dy weight / dev; dx again one of terms of the size of dp w1 / dev
    w2 = 1.0 if t["weight"] is None else float(t["weight"].abs().max())
    g = grads["dy"].double().cpu().abs().amax(-1) * w2 / dev2
    dh = 4 * g + (grads["dresidual_out"].double().cpu().abs().amax(-1) if dres else 0)
    w1 = 1.0 if t["post_weight"] is None else float(t["post_weight"].abs().max())
    f = 1.0 if t["scale"] is None else float(t["scale"].abs().max())
    xhat = (u["x"].detach().abs().amax(-1) / dev1 if post else u["x"].detach().abs().amax(-1)) + 1
    dx = dh * f * w1 * (4 / dev1 if post else 1)
    sizes = dict(x=dx, residual=dh, z=dh * f * (w1 * xhat + 1), scale=dh * (w1 * xhat + 1), post_weight=dh * f * xhat, post_bias=dh * f,
                 weight=grads["dy"].double().cpu().abs().amax(-1) * r2, bias=grads["dy"].double().cpu().abs().amax(-1))
    for name in NAMES:
        got = out["d" + name]
        if t[name] is None:
            assert got is None
            continue
        per_row = t[name].dim() == 2
        steps = (300 + (0 if per_row else rows)) * first * r2
        size = float(sizes[name].max()) * (1 if per_row else max(1.0, rows ** 0.5))
        ref.close(got, want[name], steps, label + " d" + name, scale=max(float(want[name].abs().max()), size))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [1, 2, 3, 8, 33, 64, 128, 129, 256, 257, 512, 513, 1024, 1032, 2048, 2049, 4096, 4104, 8192, 8193, 16383, 16384])
def test_sizes(lib, types, D):
    for rms, post, gate in ((True, True, True), (False, False, False), (False, True, True)):
        t, grads = inputs(types, 5, D, gate=gate, seed=D)
        if D == 1 and not rms:
            t["x"] = t["x"] * 0 + 1.0  # one column is its own mean
        check(lib, t, grads, rms, post, "D=%d rms=%s post=%s" % (D, rms, post))


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 609, 3000])
def test_rows(lib, rows):
    for D in (40, 272, 1024):
        t, grads = inputs(TYPES[1], rows, D, seed=rows)
        check(lib, t, grads, True, True, "rows=%d D=%d" % (rows, D))


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("scale", [True, False])
@pytest.mark.parametrize("weights,biases", [(True, False), (False, True), (False, False)])
def test_options(lib, gate, scale, weights, biases):
    for post in (True, False):
        for rms in (True, False):
            for D in (96, 97):
                t, grads = inputs(TYPES[2], 33, D, gate, scale, weights, biases, seed=4)
                check(lib, t, grads, rms, post, "options", dres=rms)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [520, 33, 2048])
def test_in_place(lib, types, D):
    t, grads = inputs(types, 700, D, seed=D)
    kind = dict(rms=True, post=True)
    y, h = lib.block_norm_fwd(*args(t), **kind)
    for over in ("x", "z"):
        u = {k: v.clone() for k, v in t.items()}
        y2, h2 = lib.block_norm_fwd(*args(u), **kind, y=u[over], residual_out=u["residual"])
        assert y2 is u[over] and h2 is u["residual"]
        assert torch.equal(y2, y) and torch.equal(h2, h)
    out = lib.block_norm_bwd(*args(t), **kind, **grads)
    # through the C entry point: d_x over d_y, d_residual over d_residual_out, d_z over z
    u = {k: v.clone() for k, v in t.items()}
    g = {k: v.clone() for k, v in grads.items()}
    sums = [torch.empty(D, device=DEV) for _ in range(5)]
    code, rcode = lib.dtype_code(types[0]), lib.dtype_code(types[1])
    need = lib.load().dn_block_norm_bwd_workspace_bytes(700, D, code, rcode)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    p = lambda x: x.data_ptr()
    st = lib.load().dn_block_norm_bwd(*(p(u[k]) for k in NAMES), 700, D, code, rcode, 1e-5, lib.DN_NORM_RMS | lib.DN_NORM_POST,
                                      p(g["dy"]), p(g["dresidual_out"]), p(g["dy"]), p(g["dresidual_out"]), p(u["z"]),
                                      *(p(s) for s in sums), p(ws), need, torch.cuda.current_stream().cuda_stream)
    assert st == lib.DN_OK
    for got, name in zip([g["dy"], g["dresidual_out"], u["z"]] + sums,
                         ("dx", "dresidual", "dz", "dscale", "dpost_weight", "dpost_bias", "dweight", "dbias")):
        assert torch.equal(got, out[name]), name


def test_a_bad_row_stays_a_row(lib):
    t, grads = inputs(TYPES[1], 64, 256, seed=2)
    y, h = lib.block_norm_fwd(*args(t))
    out = lib.block_norm_bwd(*args(t), **grads)
    t["x"][7, 3] = float("inf")
    t["residual"][9, 2] = float("nan")
    y2, h2 = lib.block_norm_fwd(*args(t))
    out2 = lib.block_norm_bwd(*args(t), **grads)
    rest = torch.tensor([i not in (7, 9) for i in range(64)])
    for a, b in ((y, y2), (h, h2), (out["dx"], out2["dx"]), (out["dresidual"], out2["dresidual"]), (out["dz"], out2["dz"])):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(y2[9]).all()


def test_no_rows(lib):
    t, grads = inputs(TYPES[0], 0, 64)
    y, h = lib.block_norm_fwd(*args(t))
    assert y.shape == h.shape == (0, 64)
    out = lib.block_norm_bwd(*args(t), **grads)
    assert all((out["d" + k] == 0).all() for k in NAMES[3:])


def test_gradient_by_differences(lib):
    t, grads = inputs(TYPES[2], 17, 96, seed=3)
    out = lib.block_norm_bwd(*args(t), **grads)
    for name in NAMES:
        way = normal(torch.Generator().manual_seed(5), *t[name].shape)
        loss = []
        for s in (1, -1):
            u = dict(t)
            u[name] = t[name] + s * 1e-2 * way
            y, h = lib.block_norm_fwd(*args(u))
            loss.append((y.double() * grads["dy"].double()).sum() + (h.double() * grads["dresidual_out"].double()).sum())
        diff = float(loss[0] - loss[1]) / 2e-2
        along = float((out["d" + name].double() * way.double()).sum())
        assert abs(diff - along) <= 1e-2 * float(out["d" + name].norm() * way.norm()), name
