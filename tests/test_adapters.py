"""pw_adapters against float64, its refusals, and the run norm -> projection
with adapters -> token log probabilities.

Tolerance of an output, with |.| taken elementwise in the two products
(V = |A| |x|, W = |scale| |B| V):
  2^-23 |y|                the additions of base and product, and the rounding,
  2^-22 (cols / 256 + 32) W   the shrink sums: a warp's chain has at most
                           cols / 256 MMA steps, then 16 warps and blocks,
  2^-22 (rank / 16 + 2) W  the expand sums, three terms each,
  2^-23 W (y fp32) or 2^-16 W (y bf16)   the terms v is split into;
a bf16 output adds its half step, 2^-8 |y|.
"""
import pytest

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


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


def make(gen, T, cols, rows, n, r, y=F32, order="mixed", ranks=True):
    d = {"x": torch.randn((T, cols), generator=gen).to(BF16),
         "a": (torch.randn((n, r, cols), generator=gen) * cols ** -0.5).to(BF16),
         "b": (torch.randn((n, rows, r), generator=gen) * 0.3).to(BF16),
         "base": torch.randn((T, rows), generator=gen).to(y),
         "scale": torch.rand(n, generator=gen) + 0.5,
         "ids": torch.randint(-1, n, (T,), generator=gen, dtype=torch.int32)}
    if ranks:
        d["ranks"] = torch.randint(0, r + 1, (n,), generator=gen, dtype=torch.int32)
        d["ranks"][0] = r
    if order == "runs":
        d["ids"] = torch.sort(torch.randint(0, T, (T,), generator=gen)).values.int() * n // max(T, 1)
        d["ids"] = (d["ids"] + 1) % n - (d["ids"] == n // 2).int() * n
        d["ids"] = d["ids"].clamp(min=-1).int()
    elif order == "same":
        d["ids"][:] = n - 1
    return {k: v.cuda() for k, v in d.items()}


def reference(d):
    """(y, tolerance) in float64"""
    x, y = d["x"].double(), d["base"].double().clone() if d.get("base") is not None else None
    T, cols = x.shape
    n, rows, r_max = d["b"].shape
    if y is None:
        y = torch.zeros((T, rows), dtype=torch.float64, device="cuda")
    W = torch.zeros_like(y)
    for i in range(n):
        on = (d["ids"] == i).nonzero()[:, 0]
        r = int(d["ranks"][i]) if d.get("ranks") is not None else r_max
        if not len(on) or not r:
            continue
        a, b = d["a"][i, :r].double(), d["b"][i, :, :r].double()
        sc = float(d["scale"][i]) if d.get("scale") is not None else 1.0
        y[on] += sc * (x[on] @ a.t() @ b.t())
        W[on] = abs(sc) * (x[on].abs() @ a.abs().t() @ b.abs().t())
    f32 = d.get("base") is None or d["base"].dtype == F32
    tol = W * (2.0 ** -22 * (cols / 256 + 32 + r_max / 16 + 2) + (2.0 ** -23 if f32 else 2.0 ** -16))
    return y, tol + y.abs() * (2.0 ** -23 if f32 else 2.0 ** -8 + 2.0 ** -16)


def check(gpu, d, **kw):
    y = gpu.add_adapters(**d, **kw)
    want, tol = reference(d)
    err = (y.double() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 17, 64, 255, 257, 600, 1024, 1100, 2500])
@pytest.mark.parametrize("order", ["mixed", "runs", "same"])
@pytest.mark.parametrize("r,y", [(16, F32), (64, BF16), (5, F32), (72, F32)])
def test_matches_float64(gpu, T, order, r, y):
    gen = torch.Generator().manual_seed(T * 100 + r)
    check(gpu, make(gen, T, 264, 200, 7, r, y, order))


@pytest.mark.gpu
@pytest.mark.parametrize("cols,rows", [(1, 1), (7, 3), (32, 33), (40, 1003), (1409, 130), (2048, 1408),
                                       (4096, 24), (136, 4096), (301, 302)])
@pytest.mark.parametrize("T", [3, 40, 2100])
@pytest.mark.parametrize("r", [1, 8, 12, 32, 256])
def test_odd_sizes(gpu, cols, rows, T, r):
    gen = torch.Generator().manual_seed(cols * 7 + rows + T + r)
    for y in (F32, BF16):
        check(gpu, make(gen, T, cols, rows, 3, r, y))


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(300, 300), (256, 1), (100, 90), (2304, 200)])
def test_many_adapters(gpu, T, n):
    gen = torch.Generator().manual_seed(T + n)
    check(gpu, make(gen, T, 128, 96, n, 8, ranks=False))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 2100])
def test_base_forms(gpu, T):
    """In place, none, no scale, no ranks, ids out of range, all without an adapter."""
    gen = torch.Generator().manual_seed(T)
    d = make(gen, T, 264, 136, 4, 16)
    want = check(gpu, d)
    base = d["base"].clone()
    assert gpu.add_adapters(**{**d, "base": base}, y=base) is base
    assert torch.equal(base, want)
    for drop in (["base"], ["scale"], ["ranks"], ["base", "scale", "ranks"]):
        e = {k: v for k, v in d.items() if k not in drop}
        check(gpu, e)
    wild = dict(d, ids=torch.where(d["ids"] < 0, 4 + torch.arange(T, device="cuda").int(), d["ids"]))
    assert torch.equal(gpu.add_adapters(**wild), want)
    none = dict(d, ids=torch.full_like(d["ids"], -1))
    assert torch.equal(gpu.add_adapters(**none), d["base"])
    e = {k: v for k, v in none.items() if k != "base"}
    assert (gpu.add_adapters(**e) == 0).all()
    e["y_type"] = BF16
    assert gpu.add_adapters(**e).dtype == BF16
    big = dict(d, ranks=torch.full_like(d["ranks"], 1000))     # taken into [0, max_rank]
    assert torch.equal(gpu.add_adapters(**big),
                       gpu.add_adapters(**{k: v for k, v in d.items() if k != "ranks"}))
    low = dict(d, ranks=torch.full_like(d["ranks"], -3))
    assert torch.equal(gpu.add_adapters(**low), d["base"])


@pytest.mark.gpu
@pytest.mark.parametrize("T,rows", [(8, 64), (64, 8), (1100, 24)])
def test_base_rows_that_overlap(gpu, T, rows):
    """A base whose rows are one element apart: y is row after row."""
    gen = torch.Generator().manual_seed(T)
    d = make(gen, T, 64, rows, 3, 8)
    d["base"] = torch.randn(T + rows - 1, generator=gen).cuda().unfold(0, rows, 1)
    assert d["base"].stride() == (1, 1)
    y = gpu.add_adapters(**d)
    assert y.is_contiguous()
    assert torch.equal(y, gpu.add_adapters(**{**d, "base": d["base"].contiguous()}))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 2100])
def test_nonfinite_values_stay_in_their_token(gpu, T):
    """NaN and infinities of a token, of an adapter or of unused ranks reach
    nobody else; an infinite v gives infinities, not NaN."""
    gen = torch.Generator().manual_seed(T)
    d = make(gen, T, 264, 72, 3, 16)
    d["ids"] = (torch.arange(T, device="cuda") % 3).int()
    d["ranks"] = torch.tensor([16, 9, 16], dtype=torch.int32, device="cuda")
    want = gpu.add_adapters(**d)
    e = {k: v.clone() for k, v in d.items()}
    e["x"][1, 3] = float("nan")
    e["a"][1, 9:] = float("nan")
    e["b"][1, :, 9:] = float("inf")
    e["b"][2, 5, 0] = float("nan")
    got = gpu.add_adapters(**e)
    same = torch.ones_like(want, dtype=torch.bool)
    same[1] = False
    same[2::3, 5] = False
    assert torch.equal(got[same], want[same])
    assert got[1].isnan().all() and got[2::3, 5].isnan().all()
    f = {k: v.clone() for k, v in d.items()}
    f["x"].zero_()
    f["x"][0, 0] = 3e38
    f["a"][0].zero_()
    f["a"][0, 0, 0] = 1e10
    f["b"][0, :, :] = 0.0
    f["b"][0, :, 0] = 1.0
    f["ranks"][0] = 1
    assert (gpu.add_adapters(**f)[0] == float("inf")).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 600, 2100])
@pytest.mark.parametrize("r,rank", [(16, 1), (16, 16), (20, 3), (64, 1), (72, 70), (256, 9)])
@pytest.mark.parametrize("y", [F32, BF16])
def test_infinite_x_or_scale_stays_infinite(gpu, T, r, rank, y):
    """No unused rank turns an infinity of x or of a scale into NaN: A and B
    are positive, so outputs are infinite with the sign of v."""
    gen = torch.Generator().manual_seed(T + r)
    d = make(gen, T, 136, 72, 2, r, y)
    d["a"], d["b"] = d["a"].abs() + 0.01, d["b"].abs() + 0.01
    d["a"][1, rank:] = -1.0
    d["b"][1, :, rank:] = float("nan")
    d["ranks"] = torch.tensor([r, rank], dtype=torch.int32, device="cuda")
    d["ids"] = (torch.arange(T, device="cuda") % 2 == 0).int()
    d["x"] = d["x"].abs()
    d["x"][0, 5] = float("inf")
    d["x"][T - 1 - (T - 1) % 2, 135] = float("-inf") if T > 2 else float("inf")
    got = gpu.add_adapters(**d)
    assert (got[0] == float("inf")).all()
    if T > 2:
        assert (got[T - 1 - (T - 1) % 2] == float("-inf")).all()
        assert got[2 if T > 600 else 1].isfinite().all()
    d["x"] = d["x"].clamp(-4, 4)
    d["scale"][1] = float("inf")
    got = gpu.add_adapters(**d)
    assert (got[::2] == float("inf")).all() and got[1::2].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 600, 2100])
@pytest.mark.parametrize("y", [F32, BF16])
@pytest.mark.parametrize("rows", [72, 37])
def test_base_keeps_its_bits(gpu, T, y, rows):
    """Tokens without an adapter, or of one with rank 0, keep base bit for
    bit, signed zeros and subnormals too (a NaN stays some NaN); also in place."""
    gen = torch.Generator().manual_seed(T + rows)
    d = make(gen, T, 64, rows, 3, 16, y, ranks=False)
    d["ranks"] = torch.tensor([0, 16, 16], dtype=torch.int32, device="cuda")
    d["ids"] = (torch.arange(T, device="cuda") // 3 % 3 - 1).int()       # none, rank 0, rank 16
    word = torch.int32 if y == F32 else torch.int16
    raw = d["base"].view(word)
    raw[:, 4:7] = torch.tensor([torch.iinfo(word).min, 1, torch.iinfo(word).min + 1], dtype=word)  # -0, +-least
    d["base"][:, 3] = float("nan")
    kept = (d["ids"] <= 0).nonzero()[:, 0]
    want = raw[kept][:, 4:].clone()
    got = gpu.add_adapters(**d)
    assert torch.equal(got.view(word)[kept][:, 4:], want)
    assert got[:, 3].isnan().all() and got[:, 4:].isfinite().all()
    gpu.add_adapters(**d, y=d["base"])
    assert torch.equal(raw[kept][:, 4:], want) and d["base"][:, 3].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 2100])
@pytest.mark.parametrize("y,pad", [(F32, 3), (F32, 8), (BF16, 5), (BF16, 4)])
def test_strides_alignment_and_gaps(gpu, T, y, pad):
    gen = torch.Generator().manual_seed(T + pad)
    d = make(gen, T, 136, 72, 4, 12, y)
    want = gpu.add_adapters(**d)
    wide = {k: torch.full((T, d[k].shape[1] + pad), 9.0, device="cuda").to(d[k].dtype)
            for k in ("x", "base")}
    for k in wide:
        wide[k][:, pad - 1:-1] = d[k]
        d[k] = wide[k][:, pad - 1:-1]
    out = torch.full((T, 72 + pad), 9.0, device="cuda").to(y)
    got = gpu.add_adapters(**d, y=out[:, 1:73])
    w, tol = reference(d)
    assert ((got.double() - w).abs() <= tol).all()
    gaps = torch.cat([out[:, :1], out[:, 73:]], 1)
    assert (gaps.float() == 9).all()
    # adapters at addresses that only their elements' size divides
    for k in ("a", "b"):
        flat = torch.empty(d[k].numel() + 1, dtype=BF16, device="cuda")
        flat[1:] = d[k].reshape(-1)
        d[k] = flat[1:].view(d[k].shape)
    assert ((gpu.add_adapters(**d).double() - w).abs() <= tol).all()


@pytest.mark.gpu
def test_repeatable_on_streams_and_in_graphs(gpu):
    gen = torch.Generator().manual_seed(2)
    d, e = make(gen, 70, 520, 264, 9, 32), make(gen, 2100, 264, 264, 5, 16)
    want, want2 = gpu.add_adapters(**d), gpu.add_adapters(**e)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got, got2 = gpu.add_adapters(**d, stream=s1), gpu.add_adapters(**e, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.add_adapters(**d)
    d["ids"].copy_(d["ids"].flip(0))
    graph.replay()
    assert torch.equal(out, gpu.add_adapters(**d))
    assert gpu.add_adapters(**{**d, "x": d["x"][:0], "base": d["base"][:0],
                               "ids": d["ids"][:0]}).shape == (0, 264)


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    gen = torch.Generator().manual_seed(4)
    d = make(gen, 2, 136, 72, 2, 16)
    d["ids"] = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    want = gpu.add_adapters(**d)
    flat = torch.empty((1 << 31) + 512, dtype=BF16, device="cuda")
    x = torch.as_strided(flat, (2, 136), (1 << 31, 1))
    x.copy_(d["x"])
    out = torch.as_strided(torch.empty((1 << 31) + 512, device="cuda"), (2, 72), (1 << 31, 1))
    assert torch.equal(gpu.add_adapters(**{**d, "x": x}, y=out), want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 9, 64])
def test_norm_projection_adapters_logprobs(gpu, oracle, T):
    """The calls in a row, as a served head runs them, against float64."""
    import numpy as np
    from any_precision_weight_pw_b200 import synth
    rng = np.random.default_rng(T)
    gen = torch.Generator().manual_seed(T)
    cols, V, b = 256, 1003, 4
    planes = synth.random_planes(rng, 8, V, cols)
    lut = np.sort(rng.normal(0, 0.1, size=(V, 1 << b)).astype(np.float16), axis=1)
    paged = gpu.repack_planes(torch.from_numpy(planes.view(np.int32)).cuda(), cols)
    codes = oracle.unpack_codes(planes, cols, b).astype(np.int64)
    W = torch.from_numpy(np.take_along_axis(lut, codes, 1).astype(np.float64)).cuda()
    d = make(gen, T, cols, V, 3, 16)
    res, w = torch.randn((T, cols), generator=gen).to(BF16).cuda(), torch.ones(cols, device="cuda").to(BF16)
    tokens = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32).cuda()

    x, _, h = gpu.add_rms_norm(d["x"], w, 1e-6, residual=res)
    z = gpu.linear(paged, torch.from_numpy(lut.view(np.int16)).cuda(), b, x, V,
                   adapters={k: d[k] for k in ("a", "b", "scale", "ranks")}, adapter_ids=d["ids"])
    lp, ent, idx, top = gpu.token_logprobs(z, tokens, n_top=5)

    d["x"] = x
    d["base"] = x.double() @ W.t()
    want, tol = reference(d)
    # the projection: fp32 sums of at most 256 exact products
    tol = tol + 2.0 ** -23 * 256 * (x.double().abs() @ W.abs().t())
    assert ((z.double() - want).abs() <= tol).all()
    full = torch.log_softmax(z.double(), 1)
    assert torch.allclose(lp.double(), full.gather(1, tokens.long()[:, None])[:, 0], atol=1e-5)
    assert torch.equal(idx.long(), torch.argsort(z, dim=1, descending=True, stable=True)[:, :5])


@pytest.mark.gpu
@pytest.mark.parametrize("cols,rows,r,y", [(264, 72, 16, F32), (64, 300, 72, F32), (1409, 130, 64, BF16)])
@pytest.mark.parametrize("kernel", ["shrink", "expand"])
@pytest.mark.parametrize("tile", [0, 5, 32])
def test_a_wait_that_gives_up_leaves_nan(gpu, monkeypatch, cols, rows, r, y, kernel, tile):
    """Failure detection without a fault: the test switches leave the products
    of one tile out, so the waits for them run out (5 ms).  Its tokens with an
    adapter get NaN, every other token what it always gets, and the next call
    is as ever."""
    gen = torch.Generator().manual_seed(tile)
    T = 2100
    d = make(gen, T, cols, rows, 3, r, y, ranks=False)
    d["ids"] = (torch.arange(T, device="cuda") // 50 % 4 - 1).int()     # long runs: order is kept
    want = gpu.add_adapters(**d)
    torch.cuda.synchronize()
    monkeypatch.setenv("PW_TEST_WAIT_US", "5000")
    monkeypatch.setenv("PW_TEST_STALL_TILE", str(tile if kernel == "shrink" else -2 - tile))
    got = gpu.add_adapters(**d)
    torch.cuda.synchronize()
    monkeypatch.undo()
    lost = (torch.arange(T, device="cuda") // 64 == tile) & (d["ids"] >= 0)
    assert lost.any() and not lost.all()
    assert got[lost].isnan().all() and torch.equal(got[~lost], want[~lost])
    assert torch.equal(gpu.add_adapters(**d), want)


def projection(gpu, T, cols=128, rows=40, bits=3):
    import numpy as np
    from any_precision_weight_pw_b200 import synth
    rng = np.random.default_rng(T)
    planes = synth.random_planes(rng, 4, rows, cols)
    lut = np.sort(rng.normal(0, 0.1, size=(rows, 1 << bits)).astype(np.float16), axis=1)
    return (gpu.repack_planes(torch.from_numpy(planes.view(np.int32)).cuda(), cols),
            torch.from_numpy(lut.view(np.int16)).cuda(), bits)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 1100])
def test_linear_refuses_adapters_before_the_projection(gpu, T):
    """A refused adapter leaves y as it was."""
    gen = torch.Generator().manual_seed(T)
    block = projection(gpu, T)
    d = make(gen, T, 128, 40, 3, 16)
    ok = {k: d[k] for k in ("a", "b", "scale", "ranks")}
    y = torch.full((T, 40), 7.0, device="cuda")
    for ad, ids in ((ok, None), (ok, d["ids"][:-1]), (ok, d["ids"].long()),
                    (dict(ok, a=ok["a"][:, :8]), d["ids"]), (dict(ok, scale=ok["scale"][:2]), d["ids"]),
                    (dict(ok, a=ok["a"][:0], b=ok["b"][:0], scale=None, ranks=None), d["ids"]),
                    (dict(ok, a=ok["a"].repeat(1, 17, 1), b=ok["b"].repeat(1, 1, 17)), d["ids"]),
                    (dict(ok, base=y), d["ids"]), (dict(a=ok["a"]), d["ids"]), (None, d["ids"])):
        with pytest.raises(gpu.PwError):
            gpu.linear(*block, d["x"], 40, y=y, adapters=ad, adapter_ids=ids)
    torch.cuda.synchronize()
    assert (y == 7).all()
    plain = gpu.linear(*block, d["x"], 40)
    want = gpu.add_adapters(d["x"], ids=d["ids"], base=plain, **ok)
    assert torch.equal(gpu.linear(*block, d["x"], 40, y=y, adapters=ok, adapter_ids=d["ids"]), want)
    assert torch.equal(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gpu.linear(*block, d["x"], 40, adapters=ok, adapter_ids=d["ids"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_linear_with_adapters_checks_x_and_y(gpu):
    gen = torch.Generator().manual_seed(7)
    block = projection(gpu, 4)
    d = make(gen, 4, 128, 40, 3, 16)
    ok = {k: d[k] for k in ("a", "b", "scale", "ranks")}
    wide = torch.zeros((4, 256), dtype=BF16, device="cuda")
    for x, y in ((d["x"], torch.empty((4, 40), dtype=BF16, device="cuda")), (d["x"], d["base"][:3]),
                 (d["x"], torch.empty((4, 44), device="cuda")[:, :40]), (wide[:, :128], None),
                 (d["x"].float(), None), (d["x"].cpu(), None), (d["x"], d["base"].cpu())):
        with pytest.raises(gpu.PwError):
            gpu.linear(*block, x, 40, y=y, adapters=ok, adapter_ids=d["ids"])


OK = dict(x=4096, x_ld=64, a=8192, b=16384, ids=32768, ranks=33024, scale=33280, n=2, r=8, T=4, cols=64,
          rows=64, base=65536, base_ld=64, y=131072, y_type=0, y_ld=64, ws=None, ws_bytes=0)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(cols=0), 1), (dict(rows=0), 1), (dict(cols=(1 << 30) + 1), 6), (dict(n=0), 1),
    (dict(n=4194304), 1), (dict(r=0), 1), (dict(r=257), 1), (dict(y_type=2), 1), (dict(y_type=3), 1),
    (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(ids=None), 1), (dict(y=None), 1),
    (dict(x_ld=-1), 1), (dict(y_ld=63), 1), (dict(base_ld=-1), 1), (dict(base=131072, base_ld=72), 1),
    (dict(x=4097), 1), (dict(a=8193), 1), (dict(ids=32770), 1), (dict(y=131074), 1),
    (dict(T=1025), 1), (dict(T=1025, ws=262144, ws_bytes=64), 1), (dict(T=1025, ws_bytes=1 << 30), 1),
    (dict(T=1025, ws=262148, ws_bytes=1 << 30), 1), (dict(ws_bytes=-1), 1), (dict(base=65538), 1), (dict(scale=33282), 1), (dict(T=0, x=None), 0),
])
def test_refusals(pw, change, status):
    L = pw.lib()
    assert L.pw_adapters(*{**OK, **change}.values(), None) == status
    if status:
        assert b"pw_adapters" in L.pw_last_error()


def test_workspace_bytes(pw):
    size = pw.lib().pw_adapters_workspace_bytes
    assert size(1, 16, 0) == 0 and size(1024, 256, 0) == 0 and size(1025, 0, 0) == 0
    assert size(1025, 16, 0) > size(1025, 16, 1) > 0
    assert size(4096, 64, 0) == 64 * (size(1088, 64, 0) // 17)


def test_workspace_tiles_are_whole_16_byte_pieces(pw):
    """The workspace is read in 16-byte pieces: every tile of it starts on one."""
    size = pw.lib().pw_adapters_workspace_bytes
    for r in range(1, 257):
        for y in (0, 1):
            tile = size(2048, r, y) - size(1984, r, y)
            assert tile > 0 and tile % 16 == 0 and size(2048, r, y) == 32 * tile


def test_binding_refuses_cpu_tensors(pw):
    with pytest.raises(pw.PwError):
        pw.add_adapters(torch.zeros((2, 8), dtype=BF16), torch.zeros((1, 4, 8), dtype=BF16),
                        torch.zeros((1, 6, 4), dtype=BF16), torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 3])
def test_sizes_past_32_bits_are_refused(gpu, big):
    gen = torch.Generator().manual_seed(0)
    d = make(gen, 1, 8, 8, 1, 4)
    for change, names in ((dict(x=d["x"].expand(big, 8)), "x: shape"),
                          (dict(b=d["b"][:, :1].expand(1, big, 4)), "b: shape")):
        with pytest.raises(gpu.PwError, match=names):
            gpu.add_adapters(**{**d, **change})


@pytest.mark.gpu
def test_binding_refusals(gpu):
    gen = torch.Generator().manual_seed(0)
    d = make(gen, 4, 64, 40, 2, 8)
    for change in (dict(ids=d["ids"].long()), dict(ids=d["ids"][:3]), dict(ids=None),
                   dict(x=d["x"].float()), dict(x=d["x"][:, :60]), dict(a=d["a"][:, :4]),
                   dict(b=d["b"].transpose(1, 2)), dict(base=d["base"][:, :39]),
                   dict(scale=d["scale"].double()), dict(ranks=d["ranks"].cpu()),
                   dict(y=torch.empty((4, 40), dtype=BF16, device="cuda")), dict(y_type=BF16)):
        with pytest.raises(gpu.PwError):
            gpu.add_adapters(**{**d, **change})
