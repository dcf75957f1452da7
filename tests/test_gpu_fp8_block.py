"""GPU parity of the block-scaled FP8, expert and block-norm operators against their 64-bit oracle.

Tolerances, from the definitions:
  * codes and scales of a quantizer: equal, bit for bit;
  * a product rounded once to a type with eps: |err| <= eps/2 |y| (1 + 2^-8) + c S, S the sum of
    its terms' magnitudes and c = (128 + 2G) 2^-23: a group's 128 products are added in fp32 (one
    truncation of 2^-23 each at most), each group's sum is multiplied by a rounded scale product
    and added (two roundings of 2^-24 and the fma's);
  * ids, offsets, order: equal; weights: a 64-bit value rounded to fp32, renormalized and scaled
    (three fp32 roundings): 2^-22 relative;
  * norms: stated at the test.
"""
import numpy as np
import pytest

from oracle import fp8_block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


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


def values(rng, shape, dtype, loud=0.01, std=1.0):
    """(CUDA tensor of `dtype`, its exact values in float64): normal, some channels 20 times."""
    v = rng.standard_normal(shape, dtype=np.float32) * std
    v = v * np.where(rng.random(shape[-1]) < loud, 20.0, 1.0).astype(np.float32)
    t = torch.from_numpy(v).to(TYPES[dtype])
    return t.cuda(), t.double().numpy()


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def gemm_bound(y, S, dtype, G):
    return torch.finfo(TYPES[dtype]).eps / 2 * np.abs(y) * (1 + 2.0 ** -8) + \
        (128 + 2 * G) * 2.0 ** -23 * S + torch.finfo(TYPES[dtype]).tiny


def assert_bits(t, want):
    assert np.array_equal(t.cpu().numpy(), want, equal_nan=t.dtype.is_floating_point)


# ------------------------------------------------------------------ quantizers


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 8192), (3, 272), (33, 128), (130, 1040),
                                 (1025, 4096), (4100, 2064)])
def test_quantize_act(apex, M, K, dtype):
    x, v = values(np.random.default_rng(M + K), (M, K), dtype)
    codes, scales = apex.quantize_act_fp8_block(x)
    want, want_s = ob.quantize_rows(v)
    assert_bits(scales, want_s)
    assert_bits(codes, want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantize_act_every_middle(apex, dtype):
    # groups whose scale is exactly 1 (largest value 448) and whose other values are the middles
    # between E4M3 neighbours, the values themselves, and the type's neighbours of the middles
    mids = (ob.TABLE[1:] + ob.TABLE[:-1]) / 2
    t = torch.tensor(np.concatenate([mids, ob.TABLE, -mids]), dtype=TYPES[dtype])
    bits = t.view(torch.int16)
    t = torch.cat([bits, bits + 1, bits - 1]).view(TYPES[dtype])
    t = t[t.abs() <= 448]
    for s in (1.0, 2.0 ** -6, 0.75):   # 0.75: quotients beside the middles, 448 * 0.75 = 336
        n = -(-t.numel() // 127)
        x = torch.zeros((n, 128), dtype=TYPES[dtype])
        x.view(-1)[:0] = 0
        flat = torch.zeros(n * 127, dtype=TYPES[dtype])
        flat[:t.numel()] = (t.double() * s).to(TYPES[dtype])
        x[:, 1:] = flat.view(n, 127)
        x[:, 0] = 448 * s
        codes, scales = apex.quantize_act_fp8_block(x.cuda())
        want, want_s = ob.quantize_rows(x.double().numpy())
        assert np.all(want_s == np.float32(s))
        assert_bits(scales, want_s)
        assert_bits(codes, want)


def test_quantize_act_random_scales_near_middles(apex):
    # quotients as near to a middle as fp16 values and fp32 scales get: x = the fp16 nearest to
    # middle * s for many scales
    rng = np.random.default_rng(3)
    mids = (ob.TABLE[1:] + ob.TABLE[:-1]) / 2
    amax = rng.integers(1, 1 << 10, 4000) * 2.0 ** rng.integers(-12, 5, 4000)
    amax = np.minimum(amax, 60000.0).astype(np.float16).astype(np.float64)
    s = ob.scale_of(amax).astype(np.float64)
    x = (mids[rng.integers(0, 126, (4000, 128))] * s[:, None]).astype(np.float16)
    x[:, 5] = amax
    codes, scales = apex.quantize_act_fp8_block(torch.from_numpy(x).cuda())
    want, want_s = ob.quantize_rows(x.astype(np.float64))
    assert_bits(scales, want_s)
    assert_bits(codes, want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantize_act_special_groups(apex, dtype):
    info = torch.finfo(TYPES[dtype])
    x = torch.randn(8, 256, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    x[0, :128] = 0                       # a zero group
    x[1, :128] = info.smallest_normal    # equal tiny values
    x[2, :128] = 0
    x[2, 7] = info.smallest_normal / 128 if dtype == "fp16" else info.tiny   # tiny and zeros
    x[3] = info.max
    x[4, 3] = float("inf")
    x[5, 200] = float("nan")
    x[6] = -x[6].abs()
    codes, scales = apex.quantize_act_fp8_block(x.cuda())
    want, want_s = ob.quantize_rows(x.double().numpy())
    assert_bits(scales, want_s)
    # (a NaN's sign is not specified)
    got = codes.cpu().numpy()
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    # -0 and 0 are one value
    assert np.array_equal(ob.decode(got[~nan]), ob.decode(want[~nan]))


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (130, 272), (3, 70, 400)])
def test_pack_weights(apex, shape, dtype):
    w, v = values(np.random.default_rng(sum(shape)), shape, dtype, std=0.02)
    codes, scales = apex.pack_weights_fp8_block(w)
    parts = [ob.quantize_blocks(m) for m in v.reshape(-1, *shape[-2:])]
    assert_bits(scales, np.stack([p[1] for p in parts]).reshape(scales.shape))
    assert_bits(codes, np.stack([p[0] for p in parts]).reshape(shape))


# ------------------------------------------------------------------ the product


def operands(rng, M, N, K):
    """Random codes (every finite code) and scales of mixed size."""
    a = rng.integers(0, 256, (M, K), dtype=np.uint8)
    w = rng.integers(0, 256, (N, K), dtype=np.uint8)
    a[(a & 0x7F) == 0x7F] = 0
    w[(w & 0x7F) == 0x7F] = 0
    G = -(-K // 128)
    sa = np.exp(rng.normal(-6, 0.5, (M, G))).astype(np.float32)
    sw = np.exp(rng.normal(-8, 0.5, (-(-N // 128), G))).astype(np.float32)
    return a, sa, w, sw


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (2, 130, 144), (7, 1000, 272), (16, 256, 512), (17, 384, 1040),
    (31, 129, 2064), (33, 257, 4096), (64, 500, 640), (65, 512, 384), (100, 300, 3200),
    (127, 127, 112), (129, 640, 896), (200, 1111, 528), (257, 520, 1024), (300, 2000, 272),
    (1030, 769, 400), (1, 8192, 2048), (16, 4096, 8192), (48, 2048, 4096), (128, 4096, 1024),
    (1078, 3841, 272), (1078, 3846, 400), (1200, 4096, 528)])   # tiles of 256 columns
def test_gemm(apex, M, N, K, dtype):
    a, sa, w, sw = operands(np.random.default_rng(M * N + K), M, N, K)
    y = torch.full((M + 1, N), 7.0, dtype=TYPES[dtype], device="cuda")   # a row behind the last
    apex.apex_gemm_fp8_block(M, N, K, *(torch.from_numpy(t).cuda() for t in (a, sa, w, sw)), y)
    ref, S = ob.gemm(a, sa, w, sw)
    got = host(y).astype(np.float64)
    assert np.all(got[M] == 7.0)
    err = np.abs(got[:M] - ref)
    bound = gemm_bound(ref, S, dtype, -(-K // 128))
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("M,N,K", [(3, 512, 400), (40, 256, 272), (300, 512, 528),
                                   (70, 301, 272), (300, 2045, 528), (150, 1406, 400)])
def test_gemm_output_aligned_to_its_elements_alone(apex, M, N, K):
    a, sa, w, sw = operands(np.random.default_rng(12), M, N, K)
    store = torch.full((M * N + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = store[1:1 + M * N].view(M, N)
    apex.apex_gemm_fp8_block(M, N, K, *(torch.from_numpy(t).cuda() for t in (a, sa, w, sw)), y)
    ref, S = ob.gemm(a, sa, w, sw)
    assert np.all(np.abs(host(y) - ref) <= gemm_bound(ref, S, "bf16", -(-K // 128)))
    assert store[0] == 7.0 and torch.all(store[1 + M * N:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(5, 300, 8192), (90, 700, 4096), (700, 5000, 1024)])
def test_gemm_repeats_to_the_bit(apex, M, N, K):
    ops = [torch.from_numpy(t).cuda() for t in operands(np.random.default_rng(1), M, N, K)]
    first = apex.gemm_fp8_block(*ops, dtype=torch.float16)
    for _ in range(5):
        assert torch.equal(apex.gemm_fp8_block(*ops, dtype=torch.float16), first)


@pytest.mark.parametrize("M", [3, 150])
def test_gemm_infinite_and_nan_rows_stay_theirs(apex, M):
    a, sa, w, sw = operands(np.random.default_rng(2), M, 200, 400)
    a[1, 7] = 0x7F
    sa[2, 1] = np.inf
    y = apex.gemm_fp8_block(*(torch.from_numpy(t).cuda() for t in (a, sa, w, sw)))
    y = host(y)
    assert np.isnan(y[1]).all() and not np.isfinite(y[2]).any()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert np.isfinite(y[keep]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (16, 777, 1040), (70, 300, 528), (333, 900, 272)])
def test_linear(apex, M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    x, v = values(rng, (M, K), dtype)
    w, wv = values(rng, (N, K), dtype, std=0.02)
    wc, ws = apex.pack_weights_fp8_block(w)
    y = apex.linear_fp8_block(x, wc, ws)
    assert y.dtype == x.dtype
    ref, S = ob.gemm(*ob.quantize_rows(v), *ob.quantize_blocks(wv))
    assert np.all(np.abs(host(y) - ref) <= gemm_bound(ref, S, dtype, -(-K // 128)))
    # and as the quantizer and the product apart
    again = apex.gemm_fp8_block(*apex.quantize_act_fp8_block(x), wc, ws, dtype=x.dtype)
    assert torch.equal(again, y)


# ------------------------------------------------------------------ routing


def check_route(apex, z, k, dtype="fp32", mask=None, bias=None, **kw):
    t = torch.from_numpy(z).to(TYPES[dtype])
    zv = t.double().numpy()
    dev = {"mask": None if mask is None else torch.from_numpy(mask).cuda(),
           "bias": None if bias is None else torch.from_numpy(bias).cuda()}
    E = z.shape[1]
    w, ids, offsets, order = apex.route_experts(t.cuda(), k, plan=True, **dev, **kw)
    rw, rids, _ = ob.route(zv, k, mask=mask, bias=None if bias is None else bias.astype(np.float64),
                           **kw)
    assert_bits(ids, rids)
    got = w.cpu().numpy().astype(np.float64)
    nan = np.isnan(rw)
    assert np.array_equal(np.isnan(got), nan)
    assert np.all(np.abs(got[~nan] - rw[~nan]) <= 2.0 ** -22 * np.abs(rw[~nan]) + 1e-44)
    ro, rr = ob.plan(rids, E)
    assert_bits(offsets, ro)
    assert_bits(order, rr)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,topk_groups", [
    (1, 1, 1, 1, 1), (1, 64, 8, 1, 1), (5, 33, 4, 1, 1), (130, 160, 6, 8, 3), (64, 256, 8, 8, 4),
    (37, 512, 32, 32, 16), (9, 96, 2, 3, 1), (50, 7, 7, 1, 1), (21, 8, 3, 8, 4), (1000, 60, 4, 4, 4)])
def test_route(apex, T, E, k, groups, topk_groups, score):
    rng = np.random.default_rng(T * E + k)
    z = rng.standard_normal((T, E)).astype(np.float32)
    for dtype in ("fp32", "bf16", "fp16"):
        for bias in (None, (0.1 * rng.standard_normal(E)).astype(np.float32)):
            check_route(apex, z, k, dtype=dtype, bias=bias, score=score, groups=groups,
                        topk_groups=topk_groups, renormalize=bias is not None, scale=2.5,
                        mask=rng.random(T) < 0.7 if dtype == "fp16" else None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_route_ties_go_to_the_lowest(apex, score, groups, topk_groups):
    rng = np.random.default_rng(8)
    z = rng.integers(-2, 3, (200, 64)).astype(np.float32)    # nearly every value is tied
    z[0] = 0
    for bias in (None, np.zeros(64, np.float32), np.tile(np.float32([0, 0.25]), 32)):
        check_route(apex, z, 8, score=score, groups=groups, topk_groups=topk_groups, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_route_decides_as_the_exact_scores_do(apex, score, biased, groups, topk_groups):
    # logits one fp32 ulp apart: their scores agree in fp32 as often as not
    rng = np.random.default_rng(9)
    base = rng.normal(0, 1, (300, 1)).astype(np.float32)
    steps = rng.permuted(np.tile(np.arange(48), (300, 1)), axis=1)
    z = (base.view(np.int32) + steps).astype(np.int32).view(np.float32)
    if groups > 1:
        # Two groups whose best steps have the same sum differ in worth by the second order,
        # p (47 ulp)^2 = p 2^-48 |z|^2 47^2 at most, which 64 bits cannot always tell (nor can the
        # oracle): rows whose groups at the border are within 2^-49 of each other, the error of
        # two exponentials, a quotient and a sum on each side, are left out.
        v = z.astype(np.longdouble)
        p = 1 / (1 + np.exp(-v)) if score == "sigmoid" else np.exp(v) / np.exp(v).sum(1, keepdims=True)
        worth = np.sort(np.sort(p.reshape(300, groups, -1), 2)[:, :, -2:].sum(2), 1)
        a, b = worth[:, -topk_groups], worth[:, -topk_groups - 1]
        z = z[a - b > 2.0 ** -49 * a]
        assert len(z) > 200
    check_route(apex, z, 6, score=score, groups=groups, topk_groups=topk_groups,
                bias=np.zeros(48, np.float32) if biased else None)


def test_route_near_ties_through_the_bias(apex):
    # biases that bring the scores of different logits within fp32's rounding of each other
    rng = np.random.default_rng(10)
    z = rng.normal(0, 1, (1, 64)).astype(np.float32).repeat(100, 0)
    p = 1 / (1 + np.exp(-z[0].astype(np.float64)))
    bias = (0.9 - p).astype(np.float32)
    check_route(apex, z, 8, score="sigmoid", bias=bias)
    check_route(apex, z, 8, score="sigmoid", bias=bias, groups=8, topk_groups=3)


@pytest.mark.parametrize("off", [-np.inf, np.finfo(np.float32).min, -1e9])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups", [(64, 1, 1), (64, 8, 3), (160, 8, 2), (96, 32, 9)])
def test_route_biases_that_shut_experts_out(apex, E, groups, topk_groups, score, off):
    rng = np.random.default_rng(14)
    z = rng.standard_normal((200, E)).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    bias[rng.random(E) < 0.4] = off      # some groups keep one expert or none
    bias[: E // groups] = off
    if groups == 8:
        bias[-1] = -off                  # and one that is always chosen
    check_route(apex, z, 6, score=score, bias=bias, groups=groups, topk_groups=topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_special_logits(apex, score):
    rng = np.random.default_rng(11)
    z = rng.standard_normal((8, 40)).astype(np.float32)
    z[0] = -np.inf                       # a row that is masked whole
    z[1, 3:] = -np.inf                   # fewer finite logits than choices
    z[2] = np.finfo(np.float32).min
    z[3, 5] = np.nan
    z[4] = 80.0
    z[5, ::2] = -1e30
    z[6] = np.nan
    for groups, tg in ((1, 1), (5, 2)):
        check_route(apex, z, 6, score=score, groups=groups, topk_groups=tg)
    check_route(apex, z[:6], 6, score=score, mask=np.zeros(6, bool))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score,biased,groups", [("softmax", False, 1), ("sigmoid", True, 8)])
def test_route_many_tokens(apex, score, biased, groups, dtype):
    # enough tokens for several a warp, the last run ragged
    rng = np.random.default_rng(13)
    T, E = 8195, 64
    z = rng.standard_normal((T, E)).astype(np.float32)
    check_route(apex, z, 5, dtype=dtype, score=score, groups=groups, topk_groups=max(1, groups // 2),
                bias=(0.05 * rng.standard_normal(E)).astype(np.float32) if biased else None,
                mask=rng.random(T) < 0.9, renormalize=biased)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (16, 8, 64), (333, 3, 20), (77, 5, 512),
                                   (5000, 4, 100), (16384, 8, 256), (96, 8, 512), (97, 8, 512), (1024, 8, 512),
                                   (1025, 8, 512), (8193, 8, 65), (40000, 16, 512)])
def test_plan(apex, T, k, E):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.3] = 0                       # a popular expert, repeated in a row
    if T > 10:
        ids[3] = E + 5                                      # no expert: left out
        ids[4] = -7
    for v in (ids, np.full_like(ids, -1), np.full_like(ids, E - 1)):
        offsets, order = apex.plan_experts(torch.from_numpy(v).cuda(), E)
        ro, rr = ob.plan(np.where((v < 0) | (v >= E), -1, v), E)
        assert_bits(offsets, ro)
        assert_bits(order, rr)


# ------------------------------------------------------------------ the experts' products


def moe_case(apex, rng, T, E, k, H, I, dtype, ids):
    x, v = values(rng, (T, H), dtype)
    w13, w13v = values(rng, (E, 2, I, H), dtype, loud=0, std=0.05)
    w2, w2v = values(rng, (E, H, I), dtype, loud=0, std=0.05)
    c13, s13 = apex.pack_weights_fp8_block(w13)
    c2, s2 = apex.pack_weights_fp8_block(w2)
    weights = rng.random((T, k)).astype(np.float32)
    t_ids = torch.from_numpy(ids).cuda()
    offsets, order = apex.plan_experts(t_ids, E)
    args = (x, torch.from_numpy(weights).cuda(), t_ids, offsets, order, c13, s13, c2, s2)
    ref = ob.moe(v, weights.astype(np.float64), ids, c13.cpu().numpy(), s13.cpu().numpy(),
                 c2.cpu().numpy(), s2.cpu().numpy())
    return args, ref


def assert_moe(y, ref, dtype, k):
    # each product and the sum are rounded to the type: eps/2 of every term, and of the sum; a
    # hidden value beside a rounding border may take its neighbour (2^-3 of it) where the fp32
    # sums before it round apart: about (128 + 2G) 2^-23 / 2^-4 of the values, under 1e-3 in the
    # norm.  Measured against the norm of the row.
    eps = torch.finfo(TYPES[dtype]).eps
    rms = np.sqrt((ref ** 2).mean(axis=1, keepdims=True))
    err = np.abs(host(y).astype(np.float64) - ref)
    assert np.all(err <= (eps * (k + 1) ** 0.5 + 1e-3) * (np.abs(ref) + 3 * rms) + 1e-6), \
        float((err / (rms + 1e-30)).max())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 16, 16), (1, 8, 2, 256, 128), (3, 4, 4, 144, 272), (16, 16, 4, 512, 256),
    (33, 5, 2, 400, 176), (130, 3, 2, 272, 144), (257, 7, 3, 640, 384), (600, 2, 1, 256, 512),
    (1000, 40, 6, 384, 128)])
def test_moe(apex, T, E, k, H, I, dtype):
    rng = np.random.default_rng(T + E)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    args, ref = moe_case(apex, rng, T, E, k, H, I, dtype, ids)
    assert_moe(apex.moe_mlp_fp8_block(*args), ref, dtype, k)


@pytest.mark.parametrize("T,E,k", [(40, 6, 3), (300, 4, 2)])
def test_moe_padded_repeated_and_one_sided(apex, T, E, k):
    rng = np.random.default_rng(5)
    for kind in ("padded", "none", "repeated", "one"):
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        if kind == "padded":
            ids[rng.random(T) < 0.5] = -1
            ids[0, 1] = -1                       # one choice of a token alone
        elif kind == "none":
            ids[:] = -1
        elif kind == "repeated":
            ids[:, 1] = ids[:, 0]
        else:
            ids[:] = E - 1
        args, ref = moe_case(apex, rng, T, E, k, 272, 144, "bf16", ids)
        y = apex.moe_mlp_fp8_block(*args)
        assert_moe(y, ref, "bf16", k)
        dead = (ids < 0).all(1)
        assert not host(y)[dead].any()


def test_moe_bad_tokens_stay_theirs(apex):
    rng = np.random.default_rng(6)
    T, E, k = 70, 4, 2
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    args, ref = moe_case(apex, rng, T, E, k, 256, 128, "bf16", ids)
    args[0][5, 3] = float("nan")
    args[0][9, 200] = float("inf")
    y = host(apex.moe_mlp_fp8_block(*args))
    assert np.isnan(y[5]).all() and not np.isfinite(y[9]).any()
    keep = [t for t in range(T) if t not in (5, 9)]
    assert np.isfinite(y[keep]).all()


def test_moe_offsets_that_do_not_ascend_stay_in_bounds(apex):
    # nothing is promised of the values; the kernels clamp what they index with
    rng = np.random.default_rng(7)
    ids = np.zeros((20, 2), np.int32)
    args, _ = moe_case(apex, rng, 20, 4, 2, 128, 64, "bf16", ids)
    for bad in ([0, 1 << 30, 3, 40, 40], [40, 0, 40, 0, 40], [-5, -4, 7, 90, 100]):
        a = list(args)
        a[3] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        a[4] = torch.randint(-(1 << 31), (1 << 31) - 1, (40,), device="cuda").int()
        apex.moe_mlp_fp8_block(*a)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ norms


def norm_refs(c, v):
    return ob.block_norm(v["x"], v["pre"], v.get("residual"), v.get("post"), v.get("gate"),
                         c["alpha"], 1e-6, c["offset"])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 16), (1, 8192), (3, 272), (8, 1040), (130, 2048), (5, 8208),
                                 (4, 16384), (2, 32768)])
@pytest.mark.parametrize("post,gates,residual", [(True, 1, True), (False, 0, False), (True, 0, False),
                                                 (False, "T", True)])
def test_block_norm(apex, T, H, post, gates, residual, dtype):
    rng = np.random.default_rng(T + H)
    c = {"alpha": 0.5 if residual else 1.0, "offset": 1.0 if post else 0.0}
    t, v = {}, {}
    t["x"], v["x"] = values(rng, (T, H), dtype)
    t["pre"], v["pre"] = values(rng, (H,), dtype, loud=0)
    if post:
        t["post"], v["post"] = values(rng, (H,), dtype, loud=0)
    if residual:
        t["residual"], v["residual"] = values(rng, (T, H), dtype, std=2.0)
    if gates:
        t["gate"], v["gate"] = values(rng, (T if gates == "T" else gates, H), dtype, loud=0)
    h, y, codes, scales = apex.block_norm(t["x"], t["pre"], residual=t.get("residual"),
                                          post_weight=t.get("post"), gate=t.get("gate"),
                                          alpha=c["alpha"], weight_offset=c["offset"], out="both")
    rh, ry = norm_refs(c, v)
    eps = torch.finfo(TYPES[dtype]).eps
    # fp32 before the one rounding: a mean of H squares in a tree (log2 H + 8 roundings, halved by
    # the root) and a dozen products, of each of the sum's two terms
    rel = 32 * 2.0 ** -24
    parts = np.abs(c["alpha"] * (rh - v.get("residual", 0))) + np.abs(v.get("residual", 0) + 0 * rh)
    tiny = torch.finfo(TYPES[dtype]).tiny
    assert np.all(np.abs(host(h) - rh) <= eps / 2 * np.abs(rh) * 1.01 + 4 * rel * parts + tiny)
    scale_y = np.abs(ry) + np.abs(v["pre"] + c["offset"]) * parts / np.sqrt((rh ** 2).mean(1, keepdims=True))
    assert np.all(np.abs(host(y) - ry) <= eps / 2 * np.abs(ry) * 1.01 + 8 * rel * scale_y + tiny)
    # the codes: those of a y within fp32's error of the exact one
    q = ob.rows_values(codes.cpu().numpy(), scales.cpu().numpy())
    step = np.repeat(scales.cpu().numpy().astype(np.float64), 128, axis=1)[:, :H] * 2.0 ** -10
    assert np.all(np.abs(q - ry) <= np.maximum(np.abs(ry) * 2.0 ** -4, step) * 1.001 + 8 * rel * scale_y)
    want_s = ob.scale_of(np.stack([np.abs(ry[:, g:g + 128]).max(1) for g in range(0, H, 128)], 1))
    assert np.all(np.abs(scales.cpu().numpy() - want_s) <= 2.0 ** -16 * want_s)
    # the other forms are the same values
    assert torch.equal(apex.block_norm(t["x"], t["pre"], residual=t.get("residual"),
                                       post_weight=t.get("post"), gate=t.get("gate"),
                                       alpha=c["alpha"], weight_offset=c["offset"], out="values")[1], y)
    only = apex.block_norm(t["x"], residual=t.get("residual"), post_weight=t.get("post"),
                           gate=t.get("gate"), alpha=c["alpha"], weight_offset=c["offset"],
                           out="residual")
    assert torch.equal(only[0], h) and only[1:] == (None, None, None)


def test_block_norm_in_place_zero_and_bad_rows(apex):
    rng = np.random.default_rng(0)
    x, _ = values(rng, (6, 256), "bf16")
    r, _ = values(rng, (6, 256), "bf16")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    r[0] = 0
    x[1, 4] = float("nan")
    h, y, codes, scales = apex.block_norm(x, w, residual=r, post_weight=w, out="both")
    assert not y[0].any() and not codes[0].any() and not scales[0].any()
    assert torch.isnan(y[1]).all() and torch.isnan(scales[1]).all()
    assert torch.isfinite(y[2:]).all()
    r2, y2 = r.clone(), torch.empty_like(y)
    apex.apex_block_norm(x, 6, 256, r2, w, None, 0, 1.0, w, 1e-6, 0.0, r2, y2, None, None)
    assert torch.equal(r2[2:], h[2:]) and torch.equal(y2[2:], y[2:])


# ------------------------------------------------------------------ together, and how they are called


def layer(apex, x, residual, post, pre, gate, router, c13, s13, c2, s2, dense_c, dense_s):
    """A dense projection, the norms around it, routing and the experts: as a model calls them."""
    z = apex.linear_fp8_block(x, dense_c, dense_s)
    h, y, codes, scales = apex.block_norm(z, pre, residual=residual, post_weight=post, gate=gate,
                                          alpha=0.5, out="both")
    logits = apex.gemm_fp8_block(codes, scales, *router)
    weights, ids, offsets, order = apex.route_experts(logits, 2, score="sigmoid", plan=True)
    out = apex.moe_mlp_fp8_block(y, weights, ids, offsets, order, c13, s13, c2, s2)
    return apex.block_norm(out, residual=h, out="residual")[0], ids, weights


def layer_inputs(apex, T, seed=0, H=256, I=144, E=6):
    rng = np.random.default_rng(seed)
    t = {}
    x, _ = values(rng, (T, H), "bf16")
    r, _ = values(rng, (T, H), "bf16")
    post, pre, gate = (values(rng, s, "bf16", loud=0)[0] for s in ((H,), (H,), (1, H)))
    router = apex.pack_weights_fp8_block(values(rng, (E, H), "bf16", std=0.1)[0])
    w13 = apex.pack_weights_fp8_block(values(rng, (E, 2, I, H), "bf16", std=0.05)[0])
    w2 = apex.pack_weights_fp8_block(values(rng, (E, H, I), "bf16", std=0.05)[0])
    dense = apex.pack_weights_fp8_block(values(rng, (H, H), "bf16", std=0.05)[0])
    return [x, r, post, pre, gate, router, *w13, *w2, *dense]


@pytest.mark.parametrize("T", [1, 37, 300])
def test_a_layer_of_them(apex, T):
    a = layer_inputs(apex, T)
    out, ids, weights = layer(apex, *a)
    # the reference, stage by stage on the operators' own roundings
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    n = lambda t: t.cpu().numpy()           # noqa: E731
    z = ob.gemm(*ob.quantize_rows(f(a[0])), n(a[10]), n(a[11]))[0]
    z = torch.from_numpy(z).bfloat16().double().numpy()
    h, y = ob.block_norm(z, f(a[3]), f(a[1]), f(a[2]), f(a[4]), 0.5)
    yb = torch.from_numpy(y).bfloat16().double().numpy()
    ref = ob.moe(yb, f(weights), n(ids), n(a[6]), n(a[7]), n(a[8]), n(a[9])) + h
    # bf16 roundings of z, y, the products, h and the sum, and E4M3 steps that they move
    err = np.linalg.norm(f(out) - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert err.max() <= 0.03, err.max()


def test_a_layer_captured_and_replayed_with_new_inputs(apex):
    a, b = layer_inputs(apex, 37, 0), layer_inputs(apex, 37, 1)
    want = [layer(apex, *a)[0].clone(), layer(apex, b[0], *a[1:])[0].clone()]
    x = a[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(apex, x, *a[1:])
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out1 = layer(apex, x, *a[1:])[0]
    with torch.cuda.graph(g2):
        out2 = layer(apex, x, *a[1:])[0]
    for src, w in ((a[0], want[0]), (b[0], want[1]), (a[0], want[0])):
        x.copy_(src)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out1, w) and torch.equal(out2, w)


def test_two_streams_at_once(apex):
    a, b = layer_inputs(apex, 300, 0), layer_inputs(apex, 64, 1)
    want = layer(apex, *a)[0], layer(apex, *b)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got.append((layer(apex, *a)[0], 0))
        with torch.cuda.stream(s2):
            got.append((layer(apex, *b)[0], 1))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for y, i in got)


def test_a_stream_argument(apex):
    x, _ = values(np.random.default_rng(0), (40, 512), "fp16")
    w = apex.pack_weights_fp8_block(values(np.random.default_rng(1), (300, 512), "fp16")[0])
    want = apex.linear_fp8_block(x, *w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = apex.linear_fp8_block(x, *w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_no_tokens(apex):
    e = lambda *s, d=torch.bfloat16: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    assert apex.quantize_act_fp8_block(e(0, 256))[0].shape == (0, 256)
    w = apex.pack_weights_fp8_block(torch.randn(64, 256, device="cuda"))
    assert apex.linear_fp8_block(e(0, 256), *w).shape == (0, 64)
    weights, ids, offsets, order = apex.route_experts(e(0, 8), 2, plan=True)
    assert ids.shape == (0, 2) and not offsets.any() and order.numel() == 0
    w13 = apex.pack_weights_fp8_block(torch.randn(8, 2, 64, 256, device="cuda"))
    w2 = apex.pack_weights_fp8_block(torch.randn(8, 256, 64, device="cuda"))
    assert apex.moe_mlp_fp8_block(e(0, 256), weights, ids, offsets, order, *w13, *w2).shape == (0, 256)
    assert apex.block_norm(e(0, 256), e(256), out="both")[0].shape == (0, 256)


def test_gpu_refusals(apex):
    x = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        apex.quantize_act_fp8_block(x.t())                    # not contiguous
    with pytest.raises(apex.ApexError) as e:
        apex.quantize_act_fp8_block(x.float())
    assert e.value.code == apex.APEX_ERR_UNSUPPORTED
    with pytest.raises(apex.ApexError) as e:
        apex.quantize_act_fp8_block(x[:, :24].contiguous())
    assert e.value.code == apex.APEX_ERR_INVALID_ARG
    with pytest.raises(apex.ApexError) as e:
        apex.quantize_act_fp8_block(x.view(-1)[4:4 + 512].view(2, 256))
    assert e.value.code == apex.APEX_ERR_ALIGNMENT
    with pytest.raises(ValueError):
        apex.linear_fp8_block(x, torch.zeros((8, 256), dtype=torch.uint8), torch.zeros(1, 2))


# ------------------------------------------------------------------ groups by their best expert


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,topk_groups", [
    (1, 160, 6, 8, 3), (777, 160, 6, 8, 3), (64, 256, 8, 8, 4), (9, 96, 2, 3, 1), (21, 8, 3, 8, 4),
    (37, 512, 32, 32, 16), (50, 64, 4, 4, 4), (8200, 64, 6, 8, 2)])
def test_route_groups_by_their_best(apex, T, E, k, groups, topk_groups, score):
    rng = np.random.default_rng(T + E)
    z = rng.standard_normal((T, E)).astype(np.float32)
    for dtype in ("fp32", "bf16", "fp16"):
        for bias in (None, (0.1 * rng.standard_normal(E)).astype(np.float32)):
            check_route(apex, z, k, dtype=dtype, bias=bias, score=score, groups=groups,
                        topk_groups=topk_groups, renormalize=bias is not None, scale=2.5,
                        mask=rng.random(T) < 0.7 if dtype == "fp16" else None, group_score="max")
    if 1 < topk_groups < groups < E and T > 40:    # the two rules are two
        both = [apex.route_experts(torch.from_numpy(z).cuda(), k, score=score, groups=groups,
                                   topk_groups=topk_groups, group_score=g)[1] for g in ("top2", "max")]
        assert not torch.equal(*both)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_by_their_best_at_ties_and_special_logits(apex, score):
    rng = np.random.default_rng(15)
    z = rng.integers(-2, 3, (200, 64)).astype(np.float32)    # nearly every value is tied
    z[0] = 0
    z[1] = -np.inf
    z[2, 3:] = -np.inf
    z[3] = np.finfo(np.float32).min
    z[4, 5] = np.nan
    z[5] = np.nan
    z[6, ::2] = -1e30
    z[7, :8] = np.nan                    # a whole group
    for bias in (None, np.zeros(64, np.float32), np.tile(np.float32([0, 0.25]), 32)):
        check_route(apex, z, 8, score=score, groups=8, topk_groups=3, bias=bias, group_score="max")
    base = rng.normal(0, 1, (300, 1)).astype(np.float32)      # logits an fp32 ulp apart
    steps = rng.permuted(np.tile(np.arange(48), (300, 1)), axis=1)
    z = (base.view(np.int32) + steps).astype(np.int32).view(np.float32)
    check_route(apex, z, 6, score=score, groups=4, topk_groups=2, group_score="max")
