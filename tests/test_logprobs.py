"""pw_token_logprobs against float64, and its refusals.

Tolerances, absolute, with c the additions of a thread's chain (V / 512 at
most, plus the vector and tree steps, 64): s carries 2^-24 c, an exponential's
2^-21 (its approximation and its rounded argument z - m, whose mean over the
softmax is below 2^4); the logarithm turns the relative error of s into an
absolute one of log p, which adds its own roundings, 2^-23 of its terms.  The
entropy adds u / s, with the same relative error.
"""
import math

import pytest

torch = pytest.importorskip("torch")

INF = math.inf
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


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


def reference(z, tokens, n_top):
    """float64 (logprob, entropy, top_idx, top_logprob) of finite or -inf logits"""
    z = z.double()
    lp = torch.log_softmax(z, 1)
    lp = torch.where(z == -INF, z, lp)
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    given = torch.zeros(len(z), dtype=torch.float64, device=z.device)
    on = tokens >= 0
    given[on] = lp[on, tokens[on].long()]
    idx = torch.argsort(z, dim=1, descending=True, stable=True)[:, :n_top]
    return given, ent, idx.int(), lp.gather(1, idx)


def check(got, want, V):
    rel = 2.0 ** -24 * (V / 512 + 64) + 2.0 ** -21
    lp, ent, idx, top = got
    w_lp, w_ent, w_idx, w_top = want
    for a, b in [(lp, w_lp), (top, w_top)]:
        if a is None:
            continue
        inf = b == -INF
        assert torch.equal(a == -INF, inf)
        a, b = a.double()[~inf], b[~inf]
        assert ((a - b).abs() <= rel + 2.0 ** -22 * b.abs()).all(), (a - b).abs().max()
    assert ((ent.double() - w_ent).abs() <= rel * (1 + 2 * w_ent) + 2.0 ** -22 * w_ent).all()
    if idx is not None:
        assert torch.equal(idx, w_idx)


def make(gen, T, V, dtype, pad=0, std=3.0):
    z = (torch.randn((T, V + pad), generator=gen) * std).to(dtype).cuda()[:, :V]
    tokens = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32).cuda()
    return z, tokens


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (2, 7), (5, 31), (2, 500), (1, 32000), (2, 4099),
                                 (64, 1003), (300, 8192), (700, 2049), (1, 131072), (9, 50021)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n_top", [0, 1, 5, 32])
def test_matches_float64(gpu, T, V, dtype, n_top):
    n_top = min(n_top, V)
    gen = torch.Generator().manual_seed(T * 200000 + V)
    z, tokens = make(gen, T, V, dtype)
    tokens[T // 2] = -1
    got = gpu.token_logprobs(z, tokens, n_top=n_top)
    check(got, reference(z, tokens, n_top), V)
    assert (got[2] is None) == (n_top == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_any_alignment(gpu, pad, dtype):
    """Rows starting at every offset from a 16-byte boundary."""
    gen = torch.Generator().manual_seed(pad)
    for V in (5, 13, 1001, 20011):
        z, tokens = make(gen, 17, V, dtype, pad)
        check(gpu.token_logprobs(z, tokens, n_top=5), reference(z, tokens, 5), V)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 200])
def test_ties_take_the_lowest_index(gpu, T):
    """Few values, so that ties cross vectors, threads and blocks; signed zeros are equal."""
    gen = torch.Generator().manual_seed(T)
    V = 40000
    z = torch.randint(-3, 1, (T, V), generator=gen).float().cuda()
    z[:, 1::2] *= 1.0
    z[0] = 0.0
    z[0, ::3] = -0.0
    z[1] = 2.5
    tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
    for n in (1, 17, 32):
        check(gpu.token_logprobs(z, tokens, n_top=n), reference(z, tokens, n), V)
        zb = z.to(BF16)
        check(gpu.token_logprobs(zb, tokens, n_top=n), reference(zb, tokens, n), V)


@pytest.mark.gpu
def test_sorted_and_clustered_rows(gpu):
    """Orders that are worst for a selection in one pass: rising and falling
    logits, and the best ones in one thread's share or all in one place."""
    V = 100003
    up = torch.arange(V, dtype=F32, device="cuda") / 4096
    z = torch.stack([up, up.flip(0), torch.zeros(V, device="cuda"), torch.zeros(V, device="cuda")])
    z[2, 8::2048] = torch.rand(len(z[2, 8::2048]), device="cuda") + 1
    z[3, 50000:50040] = 9.0
    tokens = torch.tensor([0, V - 1, 8, 50003], dtype=torch.int32, device="cuda")
    check(gpu.token_logprobs(z, tokens, n_top=32), reference(z, tokens, 32), V)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T", [6, 400])
def test_masked_rows(gpu, dtype, T):
    """-inf masks that leave nothing, one or few logits; masks of the type's lowest value."""
    gen = torch.Generator().manual_seed(T)
    V = 30011
    z, tokens = make(gen, T, V, dtype)
    z[0] = -INF
    z[1] = -INF
    z[1, 777] = 1.5
    z[2] = -INF
    z[2, 5:9000:3000] = 0.25
    z[3] = torch.finfo(dtype).min
    z[4] = torch.finfo(dtype).min
    z[4, 12345] = 2.0
    z[5, 100:] = torch.finfo(dtype).min
    tokens[1:3] = torch.tensor([777, 0], dtype=torch.int32)
    got = gpu.token_logprobs(z, tokens, n_top=8)
    check(got, reference(z, tokens, 8), V)
    assert got[0][0] == -INF and got[1][0] == 0 and got[0][1] == 0 and got[1][1] == 0
    assert got[2][0].tolist() == list(range(8))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 400])
def test_nonfinite_rows_stay_alone(gpu, T):
    gen = torch.Generator().manual_seed(T)
    V = 20000
    z, tokens = make(gen, T, V, F32)
    z[1, 4000] = math.nan
    z[2, 17] = INF
    z[2, 18] = -INF
    z[3, [5, 900]] = -torch.tensor(math.nan, device="cuda")
    want = reference(z, tokens, 4)
    lp, ent, idx, top = gpu.token_logprobs(z, tokens, n_top=4)
    rest = torch.tensor([0] + list(range(4, T)), device="cuda")
    check((lp[rest], ent[rest], idx[rest], top[rest]), [w[rest] for w in want], V)
    for r in (1, 2, 3):
        assert lp[r].isnan() and ent[r].isnan() and top[r].isnan().all()
    assert idx[1, 0] == 4000 and idx[2, 0] == 17 and idx[3, :2].tolist() == [5, 900]
    tokens[2] = 18
    assert gpu.token_logprobs(z, tokens)[0][2] == -INF


@pytest.mark.gpu
def test_large_logits_keep_their_digits(gpu):
    """A common offset changes nothing: z - m is formed exactly."""
    gen = torch.Generator().manual_seed(3)
    z = (torch.randint(-64, 64, (3, 9000), generator=gen) / 8).cuda()
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    a = gpu.token_logprobs(z, tokens, n_top=3)
    b = gpu.token_logprobs(z + 65536.0, tokens, n_top=3)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.gpu
def test_tokens_out_of_range_and_none(gpu):
    z = torch.zeros((4, 10), device="cuda")
    tokens = torch.tensor([-1, 10, -2, 9], dtype=torch.int32, device="cuda")
    lp, ent, idx, top = gpu.token_logprobs(z, tokens)
    assert lp[0] == 0 and lp[1].isnan() and lp[2].isnan() and abs(lp[3].item() + math.log(10)) < 1e-6
    lp, ent, idx, top = gpu.token_logprobs(z, n_top=10)
    assert lp is None and idx[0].tolist() == list(range(10))
    assert gpu.token_logprobs(z[:0], tokens[:0], n_top=2)[3].shape == (0, 2)


@pytest.mark.gpu
def test_streams_capture_and_two_calls(gpu):
    gen = torch.Generator().manual_seed(5)
    z, tokens = make(gen, 3, 50000, F32)
    z2, tokens2 = make(gen, 200, 30000, BF16)
    want, want2 = gpu.token_logprobs(z, tokens, n_top=9), gpu.token_logprobs(z2, tokens2, n_top=9)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = gpu.token_logprobs(z, tokens, n_top=9, stream=s1)
        got2 = gpu.token_logprobs(z2, tokens2, n_top=9, stream=s2)
    torch.cuda.synchronize()
    for a, b in zip(want + want2, got + got2):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.token_logprobs(z, tokens, n_top=9)
    z.copy_(z.flip(1))
    graph.replay()
    for a, b in zip(gpu.token_logprobs(z, tokens, n_top=9), out):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    V = 1001
    flat = torch.empty((1 << 31) + 2 * V, dtype=BF16, device="cuda")
    z = torch.as_strided(flat, (2, V), ((1 << 31) + 1, 1))
    z.copy_(torch.randn(2, V))
    tokens = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    check(gpu.token_logprobs(z, tokens, n_top=5), reference(z, tokens, 5), V)


@pytest.mark.gpu
def test_longest_row(gpu):
    """2^31 - 1 logits: indices up to the last one, ties among the last vectors."""
    V = 2 ** 31 - 1
    z = torch.full((1, V), -1.0, dtype=BF16, device="cuda")
    at = [V - 1, V - 2, V - 9, V - 8, 12345, V - 17, 0]
    z[0, at] = 2.0
    z[0, V - 3] = 3.0
    tokens = torch.tensor([V - 1], dtype=torch.int32, device="cuda")
    lp, _, idx, top = gpu.token_logprobs(z, tokens, n_top=10)
    rest = [i for i in range(20) if i not in at][:2]
    assert idx[0].tolist() == [V - 3] + sorted(at) + rest
    assert lp[0] == top[0, 1] and (top[0, 1:8] == lp[0]).all()


OK = dict(z=4096, type=0, ld=10, T=2, V=10, tokens=8192, n_top=2, lp=8704, ent=9216, idx=9728,
          top=10240)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(type=3), 1), (dict(type=-1), 1), (dict(n_top=-1), 1),
    (dict(n_top=33, V=100), 1), (dict(n_top=11), 1), (dict(ld=-1), 1), (dict(z=None), 1),
    (dict(lp=None), 1), (dict(tokens=None), 1), (dict(idx=None), 1), (dict(top=None), 1),
    (dict(z=4098), 1), (dict(z=4097, type=1), 1), (dict(tokens=8194), 1), (dict(top=10241), 1),
    (dict(T=0, z=None), 0),
])
def test_refusals(pw, change, status):
    L = pw.lib()
    assert L.pw_token_logprobs(*{**OK, **change}.values(), None) == status
    if status:
        assert b"pw_token_logprobs" in L.pw_last_error()


def test_binding_refuses_cpu_tensors(pw):
    with pytest.raises(pw.PwError):
        pw.token_logprobs(torch.zeros(2, 8))


@pytest.mark.gpu
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 3])
def test_sizes_past_32_bits_are_refused(gpu, big):
    z = torch.zeros((1, 8), device="cuda")
    with pytest.raises(gpu.PwError):
        gpu.token_logprobs(z[:, :1].expand(big, 1))
    with pytest.raises(gpu.PwError):
        gpu.token_logprobs(z, n_top=big)


@pytest.mark.gpu
def test_binding_refusals(gpu):
    z = torch.zeros((4, 64), device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    for args, kw in [((z, t.long()), {}), ((z, t[:3]), {}), ((z, t.cpu()), {}), ((z.double(), t), {}),
                     ((z.t(), None), {}), ((z, t), dict(n_top=33)), ((z, t), dict(n_top=-1)),
                     ((z, None), dict(logprob=z[:, 0].clone())), ((z, t), dict(top_idx=t[:, None])),
                     ((z, t), dict(n_top=1, top_idx=t[:, None].float()))]:
        with pytest.raises(gpu.PwError):
            gpu.token_logprobs(*args, **kw)
