"""The experts' products against a bound that follows every rounding on the way, on the GPU.

The oracle's values are exact for the operands; the kernels differ from them by
  * a product's fp32 sums: (128 + 2G) 2^-23 of the sum of its terms' magnitudes (a group's 128
    products are added in fp32, one truncation of 2^-23 each at most; each group's sum is multiplied
    by a rounded scale product and added);
  * the hidden values' function: |silu'(z)| < 1.1 and <= sigmoid(z) (1 + |z|), which grows with z
    below 0, and 2^-20 of the value for its own evaluation
    (an exponential of 2 ulp, an addition, a reciprocal of 1 ulp, three products; where the
    exponential is subnormal, the least, 2^-149, counts against it: below 2^-20 of values above
    2^-127);
  * their E4M3 codes: a code moves to its neighbour where the error reaches a border, and the
    group's scale moves with its largest value (half an ulp of its own rounding);
  * the second product's fp32 sums, the weighted sum of k terms in fp32, and one rounding to the
    output's type: half of its eps.
Nothing is rounded to 16 bits before the last step.
"""
import numpy as np
import pytest

from oracle import fp8_block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def apex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import group_quantized_w4a4_b200 as m
    m.load_library()
    return m


@pytest.fixture(autouse=True)
def no_device_errors(apex):
    yield
    torch.cuda.synchronize()
    assert apex.apex_get_device_status() == 0


def host(t):
    return t.double().cpu().numpy()


def sums_error(K):
    return (128 + 2 * -(-K // 128)) * 2.0 ** -23


def per_group(v, reduce):
    """A value for each group of 128 columns, repeated over them."""
    g = np.stack([reduce(v[:, i:i + 128], axis=1) for i in range(0, v.shape[1], 128)], axis=1)
    return np.repeat(g, 128, axis=1)[:, :v.shape[1]]


def hidden(xv, w1, w3):
    """(values, bound of their error) of an expert's hidden rows, after the E4M3 rounding."""
    c = sums_error(xv.shape[1])
    g, u = xv @ w1.T, xv @ w3.T
    eg, eu = c * (np.abs(xv) @ np.abs(w1).T), c * (np.abs(xv) @ np.abs(w3).T)
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    h = silu * u
    with np.errstate(over="ignore"):
        slope = np.minimum(1.1, (1 + np.abs(g) + eg) / (1 + np.exp(-(g + eg))))
    eh = slope * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 2.0 ** -20 * np.abs(h)
    codes, scales = ob.quantize_rows(h)
    s = np.repeat(scales.astype(np.float64), 128, axis=1)[:, :h.shape[1]]
    top = per_group(np.abs(h), np.max)
    es = np.where(top > 0, per_group(eh, np.max) / np.where(top > 0, top, 1), 0) + 2.0 ** -23
    q = h / np.where(s > 0, s, 1)
    eq = (eh / np.where(s > 0, s, 1) + np.abs(q) * es) * 1.01
    v = ob.decode(codes)
    ev = np.maximum(np.abs(ob.decode(ob.encode(q + eq)) - v), np.abs(ob.decode(ob.encode(q - eq)) - v))
    return v * s, np.where(s > 0, ev * s * (1 + es) + np.abs(v) * s * es, 0)


def moe_bounded(x, weights, ids, w13, s13, w2, s2, dtype):
    """(y, bound) for x [T, H] in 64 bits, codes and scales as arrays."""
    T, H = x.shape
    xv = ob.rows_values(*ob.quantize_rows(x))
    y, bound, size = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids[(ids >= 0) & (ids < w13.shape[0])]):
        t, j = np.nonzero(ids == e)
        h, eh = hidden(xv[t], *(ob.blocks_values(w13[e, n], s13[e, n]) for n in (0, 1)))
        wv = ob.blocks_values(w2[e], s2[e])
        wt = weights[t, j].astype(np.float64)[:, None]
        one = h @ wv.T
        np.add.at(y, t, wt * one)
        np.add.at(size, t, np.abs(wt * one))
        np.add.at(bound, t, np.abs(wt) * (sums_error(h.shape[1]) * (np.abs(h) @ np.abs(wv).T) +
                                          eh @ np.abs(wv).T))
    k = ids.shape[1]
    bound += 2.0 ** -23 * k * size
    info = torch.finfo(TYPES[dtype])
    return y, bound + info.eps / 2 * (np.abs(y) + bound) + info.smallest_normal * info.eps


def random_codes(gen, shape, std):
    """E4M3 codes and scales of normal weights, made on the GPU without the quantizer (its scales
    are 128 x 128 maxima; here one power of two apart at random)."""
    c = torch.randn(shape, generator=gen, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    blocks = (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128))
    s = std * torch.exp2(torch.randint(-1, 2, blocks, generator=gen, device="cuda").float())
    return c, s


def experts_case(apex, seed, T, E, k, H, I, dtype, ids, std1=None, std2=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn((T, H), generator=gen, device="cuda").to(TYPES[dtype])
    c13, s13 = random_codes(gen, (E, 2, I, H), std1 or 1.5 * H ** -0.5)
    c2, s2 = random_codes(gen, (E, H, I), std2 or I ** -0.5)
    weights = torch.rand((T, k), generator=gen, device="cuda")
    t_ids = torch.from_numpy(ids).cuda()
    return [x, weights, t_ids, *apex.plan_experts(t_ids, E), c13, s13, c2, s2]


def assert_within(apex, args, dtype, rows=None):
    x, weights, ids, _, _, c13, s13, c2, s2 = args
    y = host(apex.moe_mlp_fp8_block(*args))
    E = c13.shape[0]
    at = np.arange(len(y)) if rows is None else rows
    hid = ids.cpu().numpy()[at]
    # the experts of these rows alone come to the host
    used = np.unique(hid[(hid >= 0) & (hid < E)])
    to = np.full(E + 1, -1)
    to[used] = np.arange(len(used))
    few = [t[torch.from_numpy(used).cuda()].cpu().numpy() for t in (c13, s13, c2, s2)]
    hid = np.where((hid >= 0) & (hid < E), to[np.clip(hid, -1, E - 1)], -1)
    ref, bound = moe_bounded(host(x)[at], weights.cpu().numpy()[at], hid, *few, dtype)
    assert np.isfinite(y).all()
    err = np.abs(y[at] - ref)
    assert np.all(err <= bound), float((err / bound).max())
    return ref, bound


def choices(seed, T, E, k):
    rng = np.random.default_rng(seed)
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)


# 10 rows an expert and fewer take one kernel, more the other
@pytest.mark.parametrize("T,E,k", [(9, 6, 2), (150, 4, 2)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_moe_products_beyond_fp16s_range(apex, T, E, k, dtype):
    # an expert's product reaches 10^6 and more, its weight brings it back into range
    ids = choices(T, T, E, k)
    args = experts_case(apex, 1, T, E, k, 512, 256, dtype, ids, std2=3e4)
    args[1] *= 0.002      # (the reference's own largest output is then 2.2e4)
    ref, _ = assert_within(apex, args, dtype)
    unweighted = np.abs(ref) / args[1].double().sum(1, keepdim=True).cpu().numpy()
    assert unweighted.max() > 3e5 and np.abs(ref).max() < 65504


@pytest.mark.parametrize("T", [5, 90])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_moe_choices_that_cancel(apex, T, dtype):
    # expert 1 is expert 0 with w2 = -(1 - 2^-5) times: the sum is 2^-5 of the terms
    H, I = 272, 144
    ids = np.tile(np.int32([0, 1]), (T, 1))
    args = experts_case(apex, 2, T, 2, 2, H, I, dtype, ids)
    x, weights, _, _, _, c13, s13, c2, s2 = args
    weights[:] = 1
    c13[1], s13[1] = c13[0], s13[0]
    c2[1], s2[1] = c2[0] ^ 0x80, s2[0] * (1 - 2.0 ** -5)
    ref, bound = assert_within(apex, args, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 3, 1, 16, 16), (7, 9, 3, 144, 272), (40, 8, 4, 1040, 720), (131, 3, 2, 400, 176),
    (300, 4, 2, 528, 384), (700, 5, 3, 272, 144)])
def test_moe_bounded(apex, T, E, k, H, I, dtype):
    assert_within(apex, experts_case(apex, 3, T, E, k, H, I, dtype, choices(T, T, E, k)), dtype)


@pytest.mark.parametrize("T", [3, 60])
@pytest.mark.parametrize("gate", [-4.0, -20.0, -60.0, -87.5, -88.0])
def test_moe_silu_of_large_negative_gates(apex, gate, T):
    # sigmoid(gate) down to fp32's subnormals, beside an up value that brings the product back
    H = I = 16
    ones = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")   # noqa: E731
    up = round(-np.log2(-gate * np.exp(gate)))
    c13 = ones(1, 2, I, H)
    c13[0, 0] = 0xB8
    s13 = torch.tensor([-gate / H, 2.0 ** (up - 4)], device="cuda").view(1, 2, 1, 1)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    args = [torch.ones((T, H), dtype=torch.bfloat16, device="cuda"), torch.ones((T, 1), device="cuda"),
            ids, *apex.plan_experts(ids, 1), c13, s13, ones(1, H, I), torch.ones((1, 1, 1), device="cuda")]
    ref, _ = assert_within(apex, args, "bf16")
    assert np.all((ref < -8) & (ref > -32))


@pytest.mark.parametrize("T,E,k,H,I,rows", [
    (24, 160, 8, 4096, 1536, [0, 23]), (600, 160, 8, 4096, 1536, [5, 599]),
    (40, 8, 2, 7168, 2048, [0, 7, 39]), (100, 8, 2, 7168, 2048, [3, 99]),
    (3, 512, 32, 1024, 256, None), (400, 512, 32, 1024, 256, [0, 399]),
    (4000, 4, 2, 528, 528, [0, 1, 2000, 3998, 3999])])   # several tiles for every SM
def test_moe_experts_of_large_models(apex, T, E, k, H, I, rows):
    args = experts_case(apex, 4, T, E, k, H, I, "bf16", choices(T, T, E, k))
    assert_within(apex, args, "bf16", rows and np.array(rows))


# at most 10 rows an expert take one kernel, more the other
@pytest.mark.parametrize("T", [15, 70])
def test_moe_bad_tokens_stay_theirs_in_both_kernels(apex, T):
    ids = choices(T, T, 4, 2)
    args = experts_case(apex, 5, T, 4, 2, 256, 144, "bf16", ids)
    args[0][5, 3] = float("nan")
    args[0][9, 200] = float("inf")
    y = host(apex.moe_mlp_fp8_block(*args))
    assert np.isnan(y[5]).all() and not np.isfinite(y[9]).any()
    keep = [t for t in range(T) if t not in (5, 9)]
    assert np.isfinite(y[keep]).all()


@pytest.mark.parametrize("T", [15, 70])
def test_moe_offsets_that_do_not_ascend_stay_in_bounds_in_both_kernels(apex, T):
    # nothing is promised of the values; the kernels clamp what they index with
    S = 2 * T
    args = experts_case(apex, 6, T, 4, 2, 144, 80, "bf16", np.zeros((T, 2), np.int32))
    for bad in ([0, 1 << 30, 3, S, S], [S, 0, S, 0, S], [-5, -4, 7, S + 50, S + 60]):
        a = list(args)
        a[3] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        a[4] = torch.randint(-(1 << 31), (1 << 31) - 1, (S,), device="cuda").int()
        apex.moe_mlp_fp8_block(*a)
        torch.cuda.synchronize()
    assert_within(apex, args, "bf16")      # and the same buffers serve a right call


# 256-column tiles, three rounds of them over the SMs
@pytest.mark.parametrize("N", [8192, 8186])
def test_gemm_several_tiles_for_every_sm(apex, N):
    M, K = 1300, 2064
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    a, _ = random_codes(gen, (M, K), 1.0)
    w, sw = random_codes(gen, (N, K), 0.01)
    sa = torch.rand((M, -(-K // 128)), generator=gen, device="cuda") + 0.5
    y = torch.full((M + 1, N), 7.0, dtype=torch.float16, device="cuda")
    apex.apex_gemm_fp8_block(M, N, K, a, sa, w, sw, y)
    n = lambda t: t.cpu().numpy()    # noqa: E731
    ref, S = ob.gemm(n(a), n(sa), n(w), n(sw))
    got = host(y)
    assert np.all(got[M] == 7.0)
    info = torch.finfo(torch.float16)
    bound = sums_error(K) * S
    bound += info.eps / 2 * (np.abs(ref) + bound) + info.smallest_normal * info.eps
    err = np.abs(got[:M] - ref)
    assert np.all(err <= bound), float((err / bound).max())


# two tokens for each SM and more take other kernels than a few
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H", [16, 1040, 4096, 4112, 5008, 8192])
@pytest.mark.parametrize("post,gated,residual", [(True, True, True), (False, False, False),
                                                 (True, False, True)])
def test_block_norm_of_many_tokens(apex, H, post, gated, residual, dtype):
    T = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 4
    t = TYPES[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(H)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(t)    # noqa: E731
    x, pre = rand(T, H), rand(H)
    r = rand(T, H) if residual else None
    w = rand(H) if post else None
    g = rand(T // 4, H) if gated else None
    offset, alpha = (1.0, 0.5) if post else (0.0, 1.0)
    kw = dict(residual=r, post_weight=w, gate=g, alpha=alpha, weight_offset=offset, out="both")
    h, y, codes, scales = apex.block_norm(x, pre, **kw)
    o = [None if v is None else host(v) for v in (pre, r, w, g)]
    rh, ry = ob.block_norm(host(x), *o, alpha, 1e-6, offset)
    # fp32 before the one rounding: a mean of H squares (log2 H + 8 roundings, halved by the root)
    # and a dozen products, of each of the sum's two terms
    info, rel = torch.finfo(t), 32 * 2.0 ** -24
    parts = np.abs(rh - (0 if r is None else o[1])) + (0 if r is None else np.abs(o[1]))
    half = info.eps / 2 * 1.01
    low = info.smallest_normal * info.eps
    assert np.all(np.abs(host(h) - rh) <= half * np.abs(rh) + 4 * rel * parts + low)
    rms = np.sqrt((rh ** 2).mean(1, keepdims=True))
    size = np.abs(ry) + np.abs(o[0] + offset) * parts / rms
    assert np.all(np.abs(host(y) - ry) <= half * np.abs(ry) + 8 * rel * size + low)
    s = scales.double().cpu().numpy()
    want = ob.scale_of(np.stack([np.abs(ry[:, i:i + 128]).max(1) for i in range(0, H, 128)], 1))
    assert np.all(np.abs(s - want) <= 2.0 ** -16 * want)
    q = ob.rows_values(codes.cpu().numpy(), s)
    step = np.repeat(s, 128, axis=1)[:, :H] * 2.0 ** -10
    assert np.all(np.abs(q - ry) <= np.maximum(np.abs(ry) * 2.0 ** -4, step) * 1.001 + 8 * rel * size)
    # the same rows in a small batch: the sums' order alone is another
    few = apex.block_norm(x[:4].contiguous(), pre, **{**kw, "residual": None if r is None else r[:4].contiguous(),
                                                       "gate": None if g is None else g[:1].contiguous()})
    assert np.all(np.abs(host(few[0]) - host(h)[:4]) <= 2 * half * np.abs(rh[:4]) + 8 * rel * parts[:4] + low)
