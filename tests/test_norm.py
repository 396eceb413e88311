"""pw_add_rms_norm against float64, its refusals, and pw_moe_forward_norm
against the norm and the forward it joins.

Tolerances.  The fp32 arithmetic before the output rounding: h has one
rounding; the sum of squares has at most 32 + 10 additions in a chain, half of
whose relative error reaches rstd; square root, division and two products add
one rounding each: below 2^-24 (42 / 2 + 8) < 2^-19 relative.  On top comes half
a step of the output: 2^-8 (bf16), or for e4m3 2^-4 and 2^-10 scale below its
smallest normal.
"""
import ctypes as C

import numpy as np
import pytest

torch = pytest.importorskip("torch")

ARITH = 2.0 ** -19
EPS = 1e-6
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pw():
    from any_precision_weight_pw_b200 import binding, build
    build.build()
    return binding


@pytest.fixture(scope="module")
def gpu(pw):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return pw


def rows(gen, T, H, dtype, std=1.0, pad=0):
    t = (torch.randn((T, H + pad), generator=gen) * std).to(dtype).cuda()
    return t[:, :H]


def reference(x, w, residual=None):
    """(h, y) in float64"""
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w.double()
    return h, y


def check_e4m3(q, scales, y, group):
    T, H = y.shape
    n = -(-H // group) if group else 1
    per = group or H
    padded = torch.nn.functional.pad(y, (0, n * per - H)).view(T, n, per)
    want = (padded.abs().amax(2) / 448.0).clamp(min=2.0 ** -126)
    s = scales.double().view(T, n)
    assert ((s - want).abs() <= 2 * ARITH * want).all()
    full = s.repeat_interleave(per, 1)[:, :H]
    got = q.view(E4M3).float().double() * full
    tol = y.abs() * (2.0 ** -4 + 2 * ARITH) + full * 2.0 ** -10
    assert ((got - y).abs() <= tol).all()


SHAPES = [(1, 2048), (3, 1), (5, 7), (2, 128), (33, 136), (64, 4096), (7, 1409), (3, 8200),
          (2, 16400), (2, 32768), (130, 256), (301, 64), (4, 1000), (3, 9001), (2, 32767)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("xt,rt,wt", [(BF16, None, BF16), (BF16, BF16, BF16), (F32, BF16, F32),
                                      (BF16, F32, F32), (F32, F32, BF16), (F32, None, F32)])
@pytest.mark.parametrize("out", ["bf16", "e4m3", "e4m3_group"])
def test_matches_float64(gpu, T, H, xt, rt, wt, out):
    gen = torch.Generator().manual_seed(T * 40000 + H)
    x, w = rows(gen, T, H, xt), (torch.randn(H, generator=gen) * 0.2 + 1).to(wt).cuda()
    res = None if rt is None else rows(gen, T, H, rt, 4.0)
    group = 128 if out == "e4m3_group" else 0
    y, s, ro = gpu.add_rms_norm(x, w, EPS, residual=res, y_type=BF16 if out == "bf16" else E4M3,
                                scale_group=group)
    h, want = reference(x, w, res)
    if rt is None:
        assert ro is None
    else:
        assert torch.equal(ro, (x.float() + res.float()).to(rt))
    if out == "bf16":
        assert s is None
        assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH)).all()
    else:
        check_e4m3(y, s, want, group)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(64, 4096), (2048, 4096), (300, 1409)])
@pytest.mark.parametrize("group", [0, 128])
def test_e4m3_is_the_nearest_but_at_borders(gpu, T, H, group):
    """q is e4m3(y / s) of the float64 y: only a quotient within the arithmetic's
    error of the border between two e4m3 values may fall to its other side."""
    gen = torch.Generator().manual_seed(T + H)
    x, res = rows(gen, T, H, BF16), rows(gen, T, H, BF16, 4.0)
    w = (torch.randn(H, generator=gen) * 0.2 + 1).to(BF16).cuda()
    q, s, _ = gpu.add_rms_norm(x, w, EPS, residual=res, y_type=E4M3, scale_group=group)
    _, y = reference(x, w, res)
    full = s.double().repeat_interleave(group or H, 1)[:, :H]
    exact = y / full
    low, high = ((exact * (1 + d)).clamp(-448, 448).float().to(E4M3).float() for d in (-ARITH, ARITH))
    got = q.float()
    assert ((got == low) | (got == high)).all()
    # borders are 2^-4 and more apart, so few quotients are that close to one
    assert (got != exact.clamp(-448, 448).float().to(E4M3).float()).double().mean() <= 2 * ARITH * 2 ** 4


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [3, 8])
@pytest.mark.parametrize("out,group", [(BF16, 0), (E4M3, 0), (E4M3, 128)])
def test_strided_rows_and_untouched_gaps(gpu, pad, out, group):
    """Row strides on every matrix; what lies between the rows stays."""
    gen = torch.Generator().manual_seed(pad)
    T, H = 19, 264
    x, res = rows(gen, T, H, BF16, pad=pad), rows(gen, T, H, F32, pad=pad)
    w = torch.ones(H, dtype=BF16, device="cuda")
    yb = torch.full((T, H + pad), 7.0, device="cuda").to(out)
    rb = torch.full((T, H + pad), 7.0, device="cuda")
    y, s, ro = gpu.add_rms_norm(x, w, EPS, residual=res, residual_out=rb[:, :H], y=yb[:, :H],
                                scale_group=group)
    y2, s2, ro2 = gpu.add_rms_norm(x.contiguous(), w, EPS, residual=res.contiguous(), y_type=out,
                                   scale_group=group)
    assert torch.equal(ro, ro2)
    _, want = reference(x, w, res)
    if out == BF16:
        assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH)).all()
    else:
        check_e4m3(y, s, want, group)
    assert (yb[:, H:].float() == 7).all() and (rb[:, H:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [256, 1409])
def test_in_place_and_repeated_row(gpu, H):
    gen = torch.Generator().manual_seed(H)
    x, res = rows(gen, 70, H, BF16), rows(gen, 70, H, BF16)
    w = torch.ones(H, dtype=F32, device="cuda")
    y, _, ro = gpu.add_rms_norm(x, w, EPS, residual=res)
    x2, res2 = x.clone(), res.clone()
    y2, _, ro2 = gpu.add_rms_norm(x2, w, EPS, residual=res2, residual_out=res2, y=x2)
    assert y2 is x2 and ro2 is res2
    assert torch.equal(y, x2) and torch.equal(ro, res2)
    one = x[:1].expand(5, H)                      # stride 0: one row five times
    y3, _, _ = gpu.add_rms_norm(one, w, EPS)
    y4, _, _ = gpu.add_rms_norm(x[:1].contiguous(), w, EPS)
    assert torch.equal(y3, y4.expand(5, H))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 520, 1409, 4096, 9001])
@pytest.mark.parametrize("out,group", [(BF16, 0), (E4M3, 0), (E4M3, 128)])
@pytest.mark.parametrize("columns", [1, 300, 1 << 20])
def test_products_with_large_weights(gpu, H, out, group, columns):
    """h w leaves fp32 where y does not: the first columns' weights are up to
    2^100, rows go up to 2^100 (where the squares leave fp32 as well)."""
    gen = torch.Generator().manual_seed(H + columns)
    x = (torch.randn((9, H), generator=gen) * 2.0 ** torch.arange(20, 110, 10)[:, None]).cuda()
    w = torch.randn(H, generator=gen)
    w[:columns] *= 2.0 ** 100
    w = w.cuda()
    y, s, _ = gpu.add_rms_norm(x, w, EPS, y_type=out, scale_group=group)
    _, want = reference(x, w)
    if out == BF16:
        assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH) + 2.0 ** -133).all()
    else:
        check_e4m3(y, s, want, group)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [256, 1409])
@pytest.mark.parametrize("pad", [0, 8])
def test_outputs_in_the_other_inputs_place(gpu, H, pad):
    """y in the residual's place, residual_out in x's."""
    gen = torch.Generator().manual_seed(H + pad)
    x, res = rows(gen, 70, H, BF16, pad=pad), rows(gen, 70, H, BF16, pad=pad)
    w = torch.ones(H, dtype=F32, device="cuda")
    y, _, ro = gpu.add_rms_norm(x, w, EPS, residual=res)
    gpu.add_rms_norm(x, w, EPS, residual=res, residual_out=x, y=res)
    assert torch.equal(y, res) and torch.equal(ro, x)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 520, 1409])
@pytest.mark.parametrize("out,group", [(BF16, 0), (E4M3, 0), (E4M3, 128)])
def test_zero_huge_and_nonfinite_rows(gpu, H, out, group):
    """Zeros give zeros; rows whose squares leave fp32 are as good as others;
    NaN and infinities stay in their own row."""
    gen = torch.Generator().manual_seed(H + group)
    x = rows(gen, 6, H, F32)
    x[1] = 0
    x[2] *= 1e30
    x[3] *= 1e37
    x[4, 5] = float("nan")
    x[5, 5] = float("inf")
    w = torch.ones(H, dtype=F32, device="cuda")
    y, s, _ = gpu.add_rms_norm(x, w, EPS, y_type=out, scale_group=group)
    _, want = reference(x, w)
    fine = want[:4]
    if out == BF16:
        assert ((y[:4].double() - fine).abs() <= fine.abs() * (2.0 ** -8 + ARITH)).all()
        assert y[4].isnan().all() and y[5, 5].isnan()
        assert (y[5, torch.arange(H) != 5] == 0).all()
    else:
        check_e4m3(y[:4], s[:4], fine, group)
        assert (y[1].float() == 0).all()
        assert s[4].isnan().all()
        assert s.view(6, -1)[5, 0].isnan()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(8, 64), (64, 8), (5, 130), (2, 1409)])
def test_rows_that_overlap(gpu, T, H):
    """Windows of a series: rows one element apart, outputs row after row."""
    gen = torch.Generator().manual_seed(T)
    series = torch.randn(T + H - 1, generator=gen).cuda()
    x = series.unfold(0, H, 1)
    assert x.shape == (T, H) and x.stride() == (1, 1)
    res, w = (series * 2).unfold(0, H, 1), torch.ones(H, device="cuda")
    y, _, ro = gpu.add_rms_norm(x, w, EPS, residual=res)
    y2, _, ro2 = gpu.add_rms_norm(x.contiguous(), w, EPS, residual=res.contiguous())
    assert torch.equal(y, y2) and torch.equal(ro, ro2)
    assert y.is_contiguous() and ro.is_contiguous()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 1409, 4096, 9001, 32768])
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (F32, None)])
@pytest.mark.parametrize("out,group", [(BF16, 0), (E4M3, 0), (E4M3, 128)])
@pytest.mark.parametrize("eps", [EPS, 2.0 ** 120])
def test_rows_around_the_overflow_of_squares(gpu, H, xt, rt, out, group, eps):
    """Rows from 2^48 to 2^124, so that sums of squares pass fp32's largest
    value on the way, each with a first element far below the others; eps from
    negligible to the larger term of the mean.  2^-133 is a step of the smallest
    bf16 values."""
    gen = torch.Generator().manual_seed(H)
    size = 2.0 ** torch.arange(48, 126, 2).double()
    T = len(size)
    x = torch.randn((T, H), generator=gen).clamp(-4, 4).double() * size[:, None]
    x[:, 0] = 2.0 ** -30
    x = x.to(xt).cuda()
    res = None if rt is None else (rows(gen, T, H, rt) * 0.25).to(rt)
    w = (torch.randn(H, generator=gen) * 0.2 + 1).to(BF16).cuda()
    y, s, _ = gpu.add_rms_norm(x, w, eps, residual=res, y_type=out, scale_group=group)
    h = x.double() if res is None else x.double() + res.double()
    want = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()
    if out == BF16:
        assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH) + 2.0 ** -133).all()
    else:
        check_e4m3(y, s, want, group)


@pytest.mark.gpu
def test_streams_capture_and_empty(gpu):
    gen = torch.Generator().manual_seed(1)
    x, res = rows(gen, 40, 520, BF16), rows(gen, 40, 520, BF16)
    w = torch.ones(520, dtype=BF16, device="cuda")
    want = gpu.add_rms_norm(x, w, EPS, residual=res, y_type=E4M3, scale_group=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gpu.add_rms_norm(x, w, EPS, residual=res, y_type=E4M3, scale_group=128, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.add_rms_norm(x, w, EPS, residual=res, y_type=E4M3, scale_group=128)
    x.copy_(x.flip(0))
    want = gpu.add_rms_norm(x, w, EPS, residual=res, y_type=E4M3, scale_group=128)
    graph.replay()
    for a, b in zip(want, out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    y, _, _ = gpu.add_rms_norm(x[:0], w, EPS)
    assert y.shape == (0, 520)


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    H = 264
    flat = torch.empty((1 << 31) + 2 * H, dtype=BF16, device="cuda")
    x = torch.as_strided(flat, (2, H), (1 << 31, 1))
    x.copy_(torch.randn(2, H))
    w = torch.ones(H, dtype=BF16, device="cuda")
    y, _, _ = gpu.add_rms_norm(x, w, EPS)
    y2, _, _ = gpu.add_rms_norm(x.contiguous(), w, EPS)
    assert torch.equal(y, y2)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 16])
def test_moe_forward_norm_is_norm_then_forward(gpu, T):
    from any_precision_weight_pw_b200 import synth
    layer = synth.Layer(synth.WORKLOADS["tiny_h256_f512_e8k2"], seed=0)
    dev = gpu.upload_synth_layer(layer, max_tokens=16)
    H = layer.wl.hidden
    gen = torch.Generator().manual_seed(T)
    x, res = rows(gen, T, H, BF16), rows(gen, T, H, BF16)
    w = (torch.randn(H, generator=gen) * 0.2 + 1).to(BF16).cuda()
    wr = torch.from_numpy(layer.router_w).cuda()
    n, _, ro = gpu.add_rms_norm(x, w, EPS, residual=res)
    want = dev.forward(n, wr)
    r2 = res.clone()
    y, got_ro = dev.forward_norm(x, w, EPS, wr, residual=r2, residual_out=r2)
    assert torch.equal(y, want) and torch.equal(got_ro, ro)
    n, _, _ = gpu.add_rms_norm(x, w, EPS)
    y, got_ro = dev.forward_norm(x, w, EPS, wr)
    assert torch.equal(y, dev.forward(n, wr)) and got_ro is None
    if T:
        with pytest.raises(gpu.PwError):
            dev.forward_norm(x, w, 0.0, wr)
    dev.check_device_error()
    dev.close()


OK = dict(x=4096, x_type=1, x_ld=64, res=8192, r_type=1, r_ld=64, w=16384, w_type=1, eps=1e-6, T=4,
          H=64, ro=32768, ro_ld=64, y=65536, y_type=1, y_ld=64, scales=0, group=0)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=32769), 6), (dict(x_type=2), 1), (dict(x_type=3), 1),
    (dict(r_type=2), 1), (dict(w_type=7), 1), (dict(y_type=0), 1), (dict(group=64), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(res=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1),
    (dict(y_type=3), 1), (dict(y_ld=63), 1), (dict(ro_ld=63), 1), (dict(x_ld=-64), 1),
    (dict(x=4097), 1), (dict(y=65537), 1), (dict(w=16385), 1), (dict(x_type=0, x=4098), 1),
    (dict(T=0, x=None, y=None), 0),
])
def test_refusals(pw, change, status):
    a = {**OK, **change}
    L = pw.lib()
    assert L.pw_add_rms_norm(*a.values(), None) == status
    if status:
        assert b"pw_add_rms_norm" in L.pw_last_error()


@pytest.mark.parametrize("change", [
    dict(y=4096, y_type=3, scales=131072), dict(y=4096, y_ld=72), dict(y=4096, x_type=0), dict(ro=8192, ro_ld=72),
    dict(ro=8192, r_ld=0), dict(ro=65536), dict(y=8192, y_ld=72), dict(y=8192, r_type=0),
    dict(ro=4096, ro_ld=72), dict(ro=4096, r_type=0), dict(y=4096, x_ld=0)])
def test_refuses_places_that_do_not_match(pw, change):
    """In place with another stride or type, rows would overwrite rows that are
    still to be read; two outputs in one place overwrite one another."""
    L = pw.lib()
    assert L.pw_add_rms_norm(*{**OK, **change}.values(), None) == 1
    assert b"in place" in L.pw_last_error()


@pytest.mark.parametrize("eps,status", [(2.0 ** -127, 1), (1e-40, 1), (1e-45, 1), (1e-50, 1)])
def test_refuses_subnormal_eps(pw, eps, status):
    """The squares beside such an eps would be subnormal, with few bits left."""
    assert pw.lib().pw_add_rms_norm(*{**OK, "eps": eps}.values(), None) == status


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 1409, 4096])
@pytest.mark.parametrize("out,group", [(BF16, 0), (E4M3, 0), (E4M3, 128)])
def test_least_eps(gpu, H, out, group):
    """Rows around the square root of the least eps, 2^-126: a square is off by
    2^-150 at most (half a step of the subnormals), 2^-24 of eps."""
    gen = torch.Generator().manual_seed(H)
    x = (torch.randn((12, H), generator=gen) * 2.0 ** torch.arange(-72, -48, 2)[:, None]).cuda()
    w = torch.ones(H, device="cuda")
    y, s, _ = gpu.add_rms_norm(x, w, 2.0 ** -126, y_type=out, scale_group=group)
    h = x.double()
    want = h / torch.sqrt((h * h).mean(1, keepdim=True) + 2.0 ** -126)
    if out == BF16:
        assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH)).all()
    else:
        check_e4m3(y, s, want, group)


def test_moe_forward_norm_refuses_null_handle(pw):
    assert pw.lib().pw_moe_forward_norm(None, 4096, None, 4096, 1e-6, 1, 4096, None, None, 4096,
                                        None) == 1


def layer_without_handle(pw):
    """A layer of 4 experts x 64 columns without a handle, on the CPU (-1)."""
    layer = object.__new__(pw.MoELayer)
    layer.cfg, layer._device, layer.h = dict(hidden=64, n_experts=4), -1, None
    return layer


@pytest.mark.parametrize("change,names", [
    (dict(residual=torch.zeros(3, 64, dtype=BF16)), "residual: shape"),
    (dict(x=torch.zeros(5, 63, dtype=BF16)), "x: shape"), (dict(x=torch.zeros(64, dtype=BF16)), "x: "),
    (dict(norm_weight=torch.zeros(63, dtype=BF16)), "norm_weight: shape"),
    (dict(router_w=torch.zeros(3, 64)), "router_w: shape"), (dict(bias=torch.zeros(3)), "bias: shape"),
    (dict(y=torch.zeros(4, 64, dtype=BF16)), "y: shape"),
    (dict(residual=torch.zeros(5, 64, dtype=BF16), residual_out=torch.zeros(4, 64, dtype=BF16)),
     "residual_out: shape"),
    (dict(residual=torch.zeros(5, 64)), "residual: type"), (dict(norm_weight=torch.zeros(64)), "norm_weight: type"),
    (dict(x=torch.zeros(5, 128, dtype=BF16)[:, ::2]), "x: must be contiguous"),
    (dict(residual_out=torch.zeros(5, 64, dtype=BF16)), "residual_out: needs a residual"),
    (dict(norm_weight=None), "are needed"), (dict(router_w=None), "are needed"),
])
def test_moe_forward_norm_checks_its_tensors(pw, change, names):
    """Shapes, types and layouts, by tensors on the CPU; then their device."""
    a = dict(x=torch.zeros(5, 64, dtype=BF16), norm_weight=torch.zeros(64, dtype=BF16), eps=EPS,
             router_w=torch.zeros(4, 64))
    with pytest.raises(pw.PwError) as e:
        layer_without_handle(pw).forward_norm(**{**a, **change})
    assert e.value.status == 1 and names in str(e.value)
    layer = layer_without_handle(pw)
    layer._device = 0
    with pytest.raises(pw.PwError, match="x: on another device"):
        layer.forward_norm(**a)


def test_binding_refuses_cpu_tensors(pw):
    with pytest.raises(pw.PwError):
        pw.add_rms_norm(torch.zeros(2, 8), torch.ones(8), EPS)


@pytest.mark.gpu
def test_moe_forward_norm_outputs_need_two_places(gpu):
    from any_precision_weight_pw_b200 import synth
    layer = synth.Layer(synth.WORKLOADS["tiny_h256_f512_e8k2"], seed=0)
    dev = gpu.upload_synth_layer(layer, max_tokens=16)
    H = layer.wl.hidden
    x, w = torch.ones((3, H), dtype=BF16, device="cuda"), torch.ones(H, dtype=BF16, device="cuda")
    wr, out = torch.from_numpy(layer.router_w).cuda(), torch.full((3, H), 7.0, dtype=BF16, device="cuda")
    with pytest.raises(gpu.PwError, match="two places"):
        dev.forward_norm(x, w, EPS, wr, residual=x, residual_out=out, y=out)
    torch.cuda.synchronize()
    assert (out == 7).all()
    want = dev.forward_norm(x, w, EPS, wr, residual=x)
    x2 = x.clone()
    assert dev.forward_norm(x2, w, EPS, wr, residual=x, residual_out=out, y=x2)[0] is x2
    assert torch.equal(x2, want[0]) and torch.equal(out, want[1])
    dev.close()


@pytest.mark.gpu
def test_moe_forward_norm_refusals_and_streams(gpu):
    """Types, devices and layouts are refused before anything runs; on another
    stream the outputs are the same."""
    from any_precision_weight_pw_b200 import synth
    layer = synth.Layer(synth.WORKLOADS["tiny_h256_f512_e8k2"], seed=0)
    dev = gpu.upload_synth_layer(layer, max_tokens=16)
    H = layer.wl.hidden
    gen = torch.Generator().manual_seed(1)
    a = dict(x=rows(gen, 5, H, BF16), norm_weight=torch.ones(H, dtype=BF16, device="cuda"), eps=EPS,
             router_w=torch.from_numpy(layer.router_w).cuda(), residual=rows(gen, 5, H, BF16))
    want = dev.forward_norm(**a)
    before = a["residual"].clone()
    for change in (dict(x=a["x"].float()), dict(x=a["x"].cpu()), dict(residual=a["residual"][:4]),
                   dict(residual=a["residual"].half()), dict(norm_weight=a["norm_weight"].float()),
                   dict(norm_weight=a["norm_weight"][:-1]), dict(router_w=a["router_w"].to(BF16)),
                   dict(router_w=a["router_w"].t().contiguous().t()), dict(bias=a["router_w"][0]),
                   dict(x=rows(gen, 5, H, BF16, pad=8)), dict(y=torch.empty(5, H, device="cuda")),
                   dict(residual=None, residual_out=a["x"]), dict(router_w=None), dict(eps=0.0),
                   dict(x=rows(gen, 17, H, BF16), residual=None)):
        b = {**a, **change}
        if b["residual"] is a["residual"]:
            b["residual_out"] = a["residual"]
        with pytest.raises(gpu.PwError):
            dev.forward_norm(**b)
    torch.cuda.synchronize()
    assert torch.equal(a["residual"], before)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dev.forward_norm(**a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dev.check_device_error()
    dev.close()


def test_row_checks_know_32_bits(pw):
    pw._bind()
    for shape in ((2 ** 31, 1), (2 ** 32 + 3, 1), (1, 2 ** 31)):
        with pytest.raises(pw.PwError, match="below 2"):
            pw._rows(torch.zeros(1, 1).expand(shape), "x", shape, -1, (0,))
    assert pw._rows(torch.zeros(1, 1).expand(2 ** 31 - 1, 1), "x", (2 ** 31 - 1, 1), -1, (0,)) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 3])
def test_sizes_past_32_bits_are_refused(gpu, big):
    x, w = torch.zeros((1, 8), dtype=BF16, device="cuda"), torch.ones(8, dtype=BF16, device="cuda")
    with pytest.raises(gpu.PwError):
        gpu.add_rms_norm(x[:, :1].expand(big, 1), w[:1], EPS)
    with pytest.raises(gpu.PwError):
        gpu.add_rms_norm(x, w, EPS, y_type=E4M3, scale_group=big - big % 2 ** 31)


@pytest.mark.gpu
def test_binding_refusals(gpu):
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    for args, kw in [((x, w[:63], EPS), {}), ((x, w.cpu(), EPS), {}), ((x.half(), w, EPS), {}),
                     ((x.t(), w[:4], EPS), {}), ((x, w, EPS), dict(residual=x[:3])),
                     ((x, w, EPS), dict(residual_out=x)), ((x, w, 0.0), {}),
                     ((x, w, EPS), dict(residual=x, residual_out=x.float())),
                     ((x, w, EPS), dict(y_type=F32)), ((x, w, EPS), dict(y=x.float())),
                     ((x, w, EPS), dict(scales=x[0].float())),
                     ((x, w, EPS), dict(y_type=E4M3, scale_group=64)),
                     ((x, w, EPS), dict(y_type=E4M3, scales=torch.empty(3, device="cuda")))]:
        with pytest.raises(gpu.PwError):
            gpu.add_rms_norm(*args, **kw)
