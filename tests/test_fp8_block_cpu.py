"""CPU checks of the block-scaled FP8, expert and block-norm operators: pins of their oracle, and
the argument errors, which are found on the host before anything is launched."""
import ctypes
import itertools

import numpy as np
import pytest

import group_quantized_w4a4_b200 as apex
from group_quantized_w4a4_b200 import build as apex_build
from oracle import fp8_block as ob

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    apex_build.build()
    return apex.load_library()


# ------------------------------------------------------------------ the oracle


def test_decode_is_torchs_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ob.decode(codes), want, equal_nan=True)


def test_encode_rounds_as_torch_does():
    rng = np.random.default_rng(0)
    v = np.concatenate([ob.TABLE, (ob.TABLE[1:] + ob.TABLE[:-1]) / 2,
                        np.exp(rng.uniform(np.log(1e-4), np.log(448), 20000))]).astype(np.float32)
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ob.encode(v), want)
    assert ob.encode([1e9, -1e9, np.nan]).tolist() == [0x7E, 0xFE, 0x7F]


def test_round_to_odd_keeps_the_exact_rounding():
    # the kernels round a 64-bit quotient to odd in fp32 before E4M3: the same as rounding the
    # quotient itself, here for quotients just beside every middle, where nearest fp32 is not
    mids = (ob.TABLE[1:] + ob.TABLE[:-1]) / 2
    for rel in (2.0 ** -26, -2.0 ** -26, 2.0 ** -40, -2.0 ** -40):
        q = mids * (1 + rel)
        f = q.astype(np.float32)
        toward_zero = np.where(np.abs(f.astype(np.float64)) > np.abs(q),
                               np.nextafter(f, np.float32(0)), f)
        odd = (toward_zero.view(np.uint32) | (toward_zero.astype(np.float64) != q)).view(np.float32)
        assert np.array_equal(ob.encode(odd), ob.encode(q))
        even = np.arange(126) % 2 == 0
        assert np.array_equal(ob.encode(q), np.arange(126) + (rel > 0)) and even.any()


def test_near_middle_test_covers_every_middle():
    # the kernel's bit test: every middle, and every fp32 value within 4 ulp of it, is seen
    mids = ((ob.TABLE[1:] + ob.TABLE[:-1]) / 2).astype(np.float32).view(np.uint32).astype(np.int64)
    for d in range(-4, 5):
        b = mids + d
        shift = np.where(b >= 0x3C800000, 0x80004, 4)
        # (the lowest middle, 2^-10, lies a binade above the test's lower end 2^-11)
        assert np.all((((b + shift) & 0xFFFFF) <= 8) & (b >= 0x3A000000)), d


def test_scale_by_a_residual_step_is_the_division():
    # the kernels form a / 448 as q0 = fl(a * fl(1/448)), then q0 + fl(1/448) * (a - 448 q0) in two
    # fmas; every mantissa (the operations scale with powers of two)
    a = np.arange(1 << 23, 1 << 24, dtype=np.float64) * 2.0 ** -23
    k = np.float64(np.float32(1) / np.float32(448))
    q0 = (a * k).astype(np.float32).astype(np.float64)
    residual = a - 448.0 * q0                     # exact: at most 34 bits
    assert np.array_equal(residual.astype(np.float32), residual)
    s = (residual.astype(np.longdouble) * k + q0).astype(np.float32)
    assert np.array_equal(s, a.astype(np.float32) / np.float32(448))


def test_two_bounds_and_the_middle_settle_every_rounding():
    # the kernels' rule in numpy: codes of x r (1 - 2^-21) and x r (1 + 2^-21) that agree are the
    # quotient's; where they do not, t = fl(x r) within 4 ulp of a middle is replaced by the middle
    # or its neighbour on the side of x - m s, and others round as they are.  r: 1/s and its
    # neighbours (an approximate reciprocal is within an ulp).
    rng = np.random.default_rng(4)
    n = 1 << 19
    f32 = np.float32
    x = rng.standard_normal(n).astype(np.float16).astype(f32)
    amax = np.maximum(np.abs(x), np.abs(rng.standard_normal(n) * 3).astype(np.float16).astype(f32))
    amax[::4] = np.abs(x[::4]) * rng.integers(1, 9, n // 4)       # quotients 448 / 1..8: ties too
    mids = ((ob.TABLE[1:] + ob.TABLE[:-1]) / 2).astype(f32)
    s = ob.scale_of(amax)
    x[1::4] = (mids[rng.integers(0, 126, n // 4)] * s[1::4]).astype(np.float16).astype(f32)
    x = np.where(np.abs(x) > amax, amax, x).astype(f32)
    keep = (s > 2.0 ** -100) & (x != 0)
    x, s = x[keep], s[keep]
    exact = ob.encode(x.astype(np.float64) / s.astype(np.float64))
    for step in (-1, 0, 1):
        r = (1 / s.astype(np.float64)).astype(f32)
        r = (r.view(np.int32) + step).view(f32)
        lo, hi = (ob.encode((x * (r * f32(1 + d))).astype(f32)) for d in (-2.0 ** -21, 2.0 ** -21))
        agree = lo == hi
        assert np.array_equal(lo[agree], exact[agree])
        assert 0.5 < agree.mean() < 1
        t = (x * r).astype(f32)
        b = np.abs(t).view(np.int32).astype(np.int64)
        near = (((b + np.where(b >= 0x3C800000, 0x80004, 4)) & 0xFFFFF) <= 8) & (b >= 0x3A000000)
        m = np.where(b >= 0x3C800000, (b & 0xFFF00000) | 0x80000, (b + 4) & 0xFFF00000)
        e = np.abs(x).astype(np.float64) - m.astype(np.int32).view(f32).astype(np.float64) * s
        m = np.where(near, m + np.sign(e).astype(np.int64), b).astype(np.int32).view(f32)
        settled = ob.encode(np.copysign(m, t).astype(np.float64))
        assert np.array_equal(settled, exact)


def test_quantizer_oracle_bounds():
    x = np.random.default_rng(1).standard_normal((5, 300))
    codes, s = ob.quantize_rows(x)
    v = ob.rows_values(codes, s)
    big = np.repeat(s, 128, axis=1)[:, :300] * 2.0 ** -9
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, big) * (1 + 1e-6))
    w_codes, w_s = ob.quantize_blocks(x)
    assert w_codes.shape == x.shape and w_s.shape == (1, 3)
    assert not ob.quantize_rows(np.zeros((2, 256)))[1].any()


def test_route_oracle_by_enumeration():
    z = np.array([[0.1, 2.0, -1.0, 2.0, 0.3, 0.2]])
    w, ids, p = ob.route(z, 2)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, 0.5)
    # groups {0,1} {2,3} {4,5}: the two best by the sum of their two largest
    _, ids, p = ob.route(z, 3, bias=np.array([0, 0, 9.0, 0, 0, 0]), groups=3, topk_groups=2,
                         score="sigmoid")
    assert ids.tolist() == [[2, 1, 3]]
    best = max(itertools.combinations(range(6), 2), key=lambda c: (z[0, list(c)].sum(), -c[0]))
    assert sorted(best) == [1, 3]


def test_plan_oracle():
    offsets, order = ob.plan(np.array([[2, 0], [-1, 2], [0, 0]]), 3)
    assert offsets.tolist() == [0, 3, 3, 5]
    assert order.tolist() == [1, 4, 5, 0, 3, -1]


# ------------------------------------------------------------------ refusals at the C entry


def P(v):
    return ctypes.c_void_p(v) if v else None


INVALID, UNSUPPORTED, ALIGN = (apex.APEX_ERR_INVALID_ARG, apex.APEX_ERR_UNSUPPORTED,
                               apex.APEX_ERR_ALIGNMENT)


@pytest.mark.parametrize("change,code", [
    ({"M": 0}, INVALID), ({"N": -1}, INVALID), ({"K": 200}, INVALID), ({"K": 0}, INVALID),
    ({"K": 1 << 21}, UNSUPPORTED), ({"N": 1 << 21}, UNSUPPORTED), ({"M": 1 << 31}, UNSUPPORTED),
    ({"dtype": 2}, UNSUPPORTED), ({"dtype": -1}, UNSUPPORTED), ({"a": 0}, INVALID),
    ({"y": 0}, INVALID), ({"sw": 0}, INVALID), ({"a": 0x1008}, ALIGN), ({"w": 0x3004}, ALIGN),
    ({"sa": 0x2002}, ALIGN), ({"y": 0x5001}, ALIGN)])
def test_gemm_refusals(lib, change, code):
    c = dict(M=4, N=8, K=256, a=0x1000, sa=0x2000, w=0x3000, sw=0x4000, dtype=0, y=0x5000) | change
    assert lib.apex_gemm_fp8_block(c["M"], c["N"], c["K"], P(c["a"]), P(c["sa"]), P(c["w"]),
                                   P(c["sw"]), c["dtype"], P(c["y"]), None) == code


@pytest.mark.parametrize("change,code", [
    ({"M": 0}, INVALID), ({"K": 24}, INVALID), ({"x": 0}, INVALID), ({"dtype": 2}, UNSUPPORTED),
    ({"x": 0x1002}, ALIGN), ({"codes": 0x2008}, ALIGN), ({"scales": 0x3002}, ALIGN)])
def test_quantizer_refusals(lib, change, code):
    c = dict(M=4, K=256, x=0x1000, dtype=1, codes=0x2000, scales=0x3000) | change
    assert lib.apex_quantize_act_fp8_block(P(c["x"]), c["dtype"], c["M"], c["K"], P(c["codes"]),
                                           P(c["scales"]), None) == code
    if "dtype" in change:
        c["dtype"] = 3      # weights may be fp32
    assert lib.apex_pack_weights_fp8_block(P(c["x"]), c["dtype"], 1, c["M"], c["K"],
                                           P(c["codes"]), P(c["scales"]), None) == code


@pytest.mark.parametrize("change,code", [
    ({"K": 8}, INVALID), ({"ws": 0}, INVALID), ({"wsb": 100}, INVALID), ({"ws": 0x6010}, ALIGN),
    ({"x": 0x1008}, ALIGN), ({"dtype": 2}, UNSUPPORTED)])
def test_linear_refusals(lib, change, code):
    c = dict(M=4, N=8, K=256, x=0x1000, dtype=0, ws=0x6000, wsb=1 << 20) | change
    assert lib.apex_linear_fp8_block(c["M"], c["N"], c["K"], P(c["x"]), c["dtype"], P(0x3000),
                                     P(0x4000), P(0x5000), P(c["ws"]), c["wsb"], None) == code


def test_workspace_sizes(lib):
    assert lib.apex_linear_fp8_block_workspace_size(4, 8, 200) == 0
    assert lib.apex_linear_fp8_block_workspace_size(4, 8, 272) >= 4 * 272 + 4 * 3 * 4
    assert lib.apex_moe_mlp_fp8_block_workspace_size(4, 8, 2, 100, 64) == 0
    assert lib.apex_moe_mlp_fp8_block_workspace_size(4, 8, 2, 64, 32) >= 4 * 64 + 8 * 32 + 16 * 64


@pytest.mark.parametrize("change,code", [
    ({"T": 0}, INVALID), ({"E": 0}, INVALID), ({"k": 0}, INVALID), ({"k": 9}, INVALID),
    ({"groups": 3}, INVALID), ({"groups": 4, "tg": 5}, INVALID), ({"tg": 0}, INVALID),
    ({"groups": 4, "tg": 1, "k": 3}, INVALID), ({"score": 2}, INVALID), ({"z": 0}, INVALID),
    ({"ids": 0}, INVALID), ({"E": 513}, UNSUPPORTED), ({"E": 64, "k": 33}, UNSUPPORTED),
    ({"E": 64, "groups": 64, "tg": 8}, UNSUPPORTED), ({"dtype": 3}, UNSUPPORTED),
    ({"z": 0x1002}, ALIGN), ({"ids": 0x3002}, ALIGN), ({"bias": 0x4002}, ALIGN)])
def test_route_refusals(lib, change, code):
    c = dict(T=4, E=8, k=2, groups=1, tg=1, score=0, z=0x1000, dtype=2, w=0x2000, ids=0x3000,
             bias=0) | change
    assert lib.apex_route_experts(P(c["z"]), c["dtype"], c["T"], c["E"], c["k"], c["score"],
                                  P(c["bias"]), c["groups"], c["tg"], 1, 1.0, None, P(c["w"]),
                                  P(c["ids"]), None) == code


@pytest.mark.parametrize("change,code", [
    ({"T": 0}, INVALID), ({"k": 0}, INVALID), ({"E": 0}, INVALID), ({"E": 600}, UNSUPPORTED),
    ({"T": 1 << 29, "k": 8}, UNSUPPORTED), ({"order": 0}, INVALID), ({"order": 0x3002}, ALIGN)])
def test_plan_refusals(lib, change, code):
    c = dict(T=4, k=2, E=8, order=0x3000) | change
    assert lib.apex_plan_experts(P(0x1000), c["T"], c["k"], c["E"], P(0x2000), P(c["order"]),
                                 None) == code


@pytest.mark.parametrize("change,code", [
    ({"T": 0}, INVALID), ({"H": 40}, INVALID), ({"I": 24}, INVALID), ({"E": 513}, UNSUPPORTED),
    ({"k": 33}, UNSUPPORTED), ({"dtype": 2}, UNSUPPORTED), ({"x": 0}, INVALID),
    ({"x": 0x1008}, ALIGN), ({"y": 0x7008}, ALIGN), ({"ws": 0x8010}, ALIGN), ({"wsb": 64}, INVALID),
    ({"H": 1 << 21}, UNSUPPORTED)])
def test_moe_refusals(lib, change, code):
    c = dict(T=4, E=8, k=2, H=64, I=32, x=0x1000, dtype=0, y=0x7000, ws=0x8000, wsb=1 << 20) | change
    p = [P(0x2000 + 0x100 * i) for i in range(8)]
    assert lib.apex_moe_mlp_fp8_block(c["T"], c["E"], c["k"], c["H"], c["I"], P(c["x"]),
                                      c["dtype"], *p, P(c["y"]), P(c["ws"]), c["wsb"], None) == code


@pytest.mark.parametrize("change,code", [
    ({"T": 0}, INVALID), ({"H": 12}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": float("nan")}, INVALID), ({"h": 0, "codes": 0}, INVALID), ({"pre": 0}, INVALID),
    ({"scales": 0}, INVALID), ({"H": 72}, INVALID), ({"gate": 0x5000, "rows": 3}, INVALID),
    ({"gate": 0x5000, "rows": 0}, INVALID), ({"H": 32784}, UNSUPPORTED), ({"dtype": 2}, UNSUPPORTED),
    ({"x": 0x1008}, ALIGN), ({"pre": 0x2004}, ALIGN), ({"codes": 0x4008}, ALIGN),
    ({"scales": 0x6002}, ALIGN)])
def test_block_norm_refusals(lib, change, code):
    c = dict(T=4, H=64, x=0x1000, dtype=0, pre=0x2000, h=0x3000, codes=0x4000, gate=0, rows=1,
             eps=1e-6, scales=0x6000) | change
    assert lib.apex_block_norm(P(c["x"]), c["dtype"], c["T"], c["H"], None, None, P(c["gate"]),
                               c["rows"], 1.0, P(c["pre"]), c["eps"], 0.0, P(c["h"]), None,
                               P(c["codes"]), P(c["scales"]), None) == code


# ------------------------------------------------------------------ refusals of the binding


def test_binding_refusals():
    x = torch.zeros((4, 256), dtype=torch.float16)
    with pytest.raises(ValueError):
        apex.quantize_act_fp8_block(x)                       # not on the GPU
    with pytest.raises(ValueError):
        apex.route_experts(torch.zeros(2, 8), 2, score="tanh")
    with pytest.raises(ValueError):
        apex.route_experts(torch.zeros(2, 8), 2, bias=torch.zeros(7))
    with pytest.raises(ValueError):
        apex.route_experts(torch.zeros(2, 8), 2, mask=torch.zeros(2))
    with pytest.raises(ValueError):
        apex.plan_experts(torch.zeros((2, 2), dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        apex.block_norm(x, out="nothing")
    with pytest.raises(ValueError):
        apex.block_norm(x, out="codes")                      # no pre_weight
    with pytest.raises(ValueError):
        apex.block_norm(x, x[0].float())
    with pytest.raises(ValueError):
        apex.linear_fp8_block(x, torch.zeros((8, 128), dtype=torch.uint8), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        apex.gemm_fp8_block(torch.zeros((4, 256), dtype=torch.uint8), torch.zeros(4, 3),
                            torch.zeros((8, 256), dtype=torch.uint8), torch.zeros(1, 2))


def test_the_library_loads_without_torch(lib):
    # as a program does that calls the C entry points on its own pointers
    import os
    import subprocess
    import sys
    code = ("import sys; sys.modules['torch'] = None\n"
            "import group_quantized_w4a4_b200 as apex\n"
            "lib = apex.load_library(build_if_missing=False)\n"
            "assert lib.apex_select_weight_group(16, 8192, 8192, 1.0, 1.0) in (128, 8192)\n"
            "assert lib.apex_linear_fp8_block_workspace_size(4, 8, 272) > 0\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=120)


@pytest.mark.parametrize("call", [
    lambda t, s: apex.quantize_act_fp8_block(t(4, 256), stream=s),
    lambda t, s: apex.pack_weights_fp8_block(t(4, 256), stream=s),
    lambda t, s: apex.gemm_fp8_block(t(4, 256), t(4, 2), t(8, 256), t(1, 2), stream=s),
    lambda t, s: apex.linear_fp8_block(t(4, 256), t(8, 256), t(1, 2), stream=s),
    lambda t, s: apex.route_experts(t(2, 8), 2, stream=s),
    lambda t, s: apex.plan_experts(t(2, 2), 4, stream=s),
    lambda t, s: apex.moe_mlp_fp8_block(*(t(2, 2) for _ in range(9)), stream=s),
    lambda t, s: apex.block_norm(t(4, 256), t(256), stream=s)])
def test_a_stream_of_another_device_is_refused(call):
    # (the device is compared before anything else is done with the stream or the tensors)
    class Elsewhere:
        device_index = 3
    with pytest.raises(ValueError, match="a stream of the tensors' device"):
        call(lambda *shape: torch.zeros(shape), Elsewhere())


def test_gemm_refuses_a_dtype_that_is_not_outs():
    a, sa, w, sw = (torch.zeros((4, 256), dtype=torch.uint8), torch.zeros(4, 2),
                    torch.zeros((8, 256), dtype=torch.uint8), torch.zeros(1, 2))
    for dtype, out in ((torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)):
        with pytest.raises(ValueError, match="out is"):
            apex.gemm_fp8_block(a, sa, w, sw, dtype=dtype, out=torch.zeros((4, 8), dtype=out))
    with pytest.raises(ValueError, match="expected fp16 or bf16"):
        apex.gemm_fp8_block(a, sa, w, sw, out=torch.zeros((4, 8)))
    for out in (torch.float16, torch.bfloat16):      # alone, out says the type: no complaint of it
        with pytest.raises(ValueError, match="CUDA tensor"):
            apex.gemm_fp8_block(a, sa, w, sw, out=torch.zeros((4, 8), dtype=out))


def test_the_torch_binding_is_of_this_torch(lib, monkeypatch):
    apex_build.build_torch()
    assert not apex_build.torch_is_stale()
    monkeypatch.setattr(torch, "__version__", "9.9.0+other")
    assert apex_build.torch_is_stale()       # another torch: built again, under another name


def test_route_oracles_two_group_rules():
    # groups {0,1} {2,3} {4,5}: the largest single score is in the last, the largest pair in the first
    z = np.array([[1.0, 0.9, 0.5, 0.4, 1.1, -9.0]])
    assert ob.route(z, 2, groups=3, topk_groups=1)[1].tolist() == [[0, 1]]
    assert ob.route(z, 2, groups=3, topk_groups=1, group_score="max")[1].tolist() == [[4, 5]]
    bias = np.array([0, 0, 0, 0.7, 0, 0])      # and by the biased score of the middle's best
    assert ob.route(z, 2, bias=bias, groups=3, topk_groups=1, group_score="max")[1].tolist() == [[3, 2]]


def test_group_rule_refusals(lib):
    with pytest.raises(ValueError, match="group_score"):
        apex.route_experts(torch.zeros(2, 8), 2, group_score="mean")
    for score, code in ((0x200, INVALID), (0x102, INVALID), (0x100, ALIGN), (0x101, ALIGN)):
        assert lib.apex_route_experts(P(0x1002), 2, 4, 8, 2, score, None, 4, 2, 1, 1.0, None,
                                      P(0x2000), P(0x3000), None) == code
