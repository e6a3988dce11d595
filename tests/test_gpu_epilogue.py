"""Products with bias, activation and residual in the epilogue.

The sharp inputs: scales that are powers of two, activations in {-1, 0, 1} and
integer zero-points, so the product is an integer multiple of the scale that
fp32 holds exactly however it is summed.  The reference is the oracle's fp64
product with the rest in fp64; the kernels may differ from it by one rounding
to the output type (eps / 2 of the value) and, for SiLU and GELU, by the fp32
evaluation of v / (1 + e^-u): 2^-20 of the value covers expf (2 ulp, 2^-22),
the argument (u up to 90 before the quotient is below 2^-100 of v: its 2^-23
relative error shifts e^-u by at most 2^-16 there, weighted with e^-u / (1 + e^-u)
where u < 0 -- so 2^-16 of the value in all) and the division."""
import numpy as np
import pytest
import torch

import workloads as wl
from _util import act_dtype, bits_to_tensor, oracle_y, repack_layer, tensor_f64, within_tolerance

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu"]


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_w4a16_amd as m
    m.lib()
    assert torch.cuda.is_available()
    return m


def activate(v, act):
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    if act == "silu":
        return v / (1 + np.exp(np.clip(-v, None, 700)))
    if act == "gelu":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


def exact_problem(M, K, N, bits, gs, mode, dt, seed, act_order=False):
    L = wl.make_layer(K, N, bits, gs, mode, seed=seed, act_order=act_order)
    rng = np.random.Generator(np.random.PCG64(seed))
    L.scales = wl.to_f16_bits(np.where(rng.random(L.scales.shape) < 0.5, 2.0 ** -5, 2.0 ** -6))
    if mode == wl.ZERO_F16:
        L.zeros = wl.to_f16_bits(rng.integers(0, 2 ** bits, L.zeros.shape).astype(np.float64))
    x = wl.to_act_bits(rng.integers(-1, 2, (M, K)).astype(np.float64), dt)
    bias = wl.to_act_bits(rng.standard_normal(N), dt)
    res = wl.to_act_bits(rng.standard_normal((M, N)) * 3, dt)
    return L, x, bias, res


def f64(bits, dt):
    return tensor_f64(bits_to_tensor(bits, act_dtype(dt), "cpu"))


def check(wq, fn, L, x, dt, y64, bias, res, act, in_place=False):
    layer = repack_layer(wq, L)
    t = lambda b: None if b is None else bits_to_tensor(b, act_dtype(dt), "cuda")
    tb, tr = t(bias), t(res)
    y = getattr(wq, fn)(t(x), layer, bias=tb, act=act, residual=tr, out=tr if in_place else None)
    if in_place:
        assert y.data_ptr() == tr.data_ptr()
    want = activate(y64 + (0 if bias is None else f64(bias, dt)), act) + (0 if res is None else f64(res, dt))
    v = np.abs(activate(y64 + (0 if bias is None else f64(bias, dt)), act))
    half = 2.0 ** -11 if dt == wl.F16 else 2.0 ** -8
    # the exact sums without a smooth activation are rounded once and nothing else (the fp32 sum of an exact value,
    # a bias and a residual rounds twice at 2^-24)
    inner = 2.0 ** -16 if act in ("silu", "gelu") else 2.0 ** -23
    bound = half * np.abs(want) + (v + np.abs(want) + np.abs(y64)) * inner + 2.0 ** -25
    err = np.abs(tensor_f64(y) - want)
    assert (err <= bound).all(), (fn, act, float((err / bound).max()))


@pytest.mark.parametrize("dt", [wl.F16, wl.BF16])
@pytest.mark.parametrize("M", [1, 4, 5, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("bits,gs,mode", [(4, 128, wl.SYM), (4, 32, wl.ZERO_F16), (3, -1, wl.ZERO_F16), (2, 256, wl.SYM)])
def test_gemv_epilogue(orc, wq, bits, gs, mode, M, dt):
    K, N = 512, 208
    L, x, bias, res = exact_problem(M, K, N, bits, gs, mode, dt, 100 * bits + M)
    y64 = oracle_y(orc, x, dt, L)
    for i, act in enumerate(ACTS):
        check(wq, "wq_gemv_epilogue", L, x, dt, y64, bias if i != 1 else None, res if i != 2 else None, act, i == 3)


@pytest.mark.parametrize("dt", [wl.F16, wl.BF16])
@pytest.mark.parametrize("M,K,N", [(33, 512, 208), (64, 512, 272), (130, 256, 208), (200, 2048, 80), (500, 256, 8208)])
@pytest.mark.parametrize("bits,gs,mode", [(4, -1, wl.SYM), (4, 128, wl.ZERO_F16), (3, 32, wl.SYM), (2, 256, wl.ZERO_F16)])
def test_gemm_epilogue(orc, wq, bits, gs, mode, M, K, N, dt):
    """Each tile shape, with the keys of K split and whole."""
    L, x, bias, res = exact_problem(M, K, N, bits, gs, mode, dt, 100 * bits + M)
    y64 = oracle_y(orc, x, dt, L)
    for i, act in enumerate(ACTS):
        check(wq, "wq_gemm_epilogue", L, x, dt, y64, bias if i != 1 else None, res if i != 2 else None, act, i == 3)


def test_gemm_epilogue_128_by_256_tiles(wq):
    """The widest tiles (480 workgroups and more), against a float64 product of the debug weights."""
    M, K, N, dt = 1000, 256, 16400, wl.F16
    for mode, gs in ((wl.SYM, -1), (wl.ZERO_F16, 128)):
        L, x, bias, res = exact_problem(M, K, N, 4, gs, mode, dt, 9)
        w = wq.wq_dequant_debug(repack_layer(wq, L), torch.float16).double()
        y64 = (bits_to_tensor(x, torch.float16, "cuda").double() @ w).cpu().numpy()
        check(wq, "wq_gemm_epilogue", L, x, dt, y64, bias, res, "gelu")
        check(wq, "wq_gemm_epilogue", L, x, dt, y64, None, res, "none", True)


@pytest.mark.parametrize("M", [1, 16, 300])
def test_epilogue_without_parts_is_the_plain_product(wq, M):
    """Nothing to add: the plain product's bits, and bits of it under act-order, through linear() too."""
    for mode, act_order in ((wl.SYM, False), (wl.ZERO_PACKED, True), (wl.LUT, False), (wl.ZERO_F16_G8, False)):
        L = wl.make_layer(1024, 160, 4, 128, mode, 5, lut=wl.nf_table(4) if mode == wl.LUT else None, act_order=act_order)
        layer = repack_layer(wq, L)
        x = bits_to_tensor(wl.make_x(M, 1024, wl.F16, 3), torch.float16, "cuda")
        fns = ("gemv", "gemm") if M <= 32 else ("gemm",)
        for fn in fns:
            assert torch.equal(getattr(wq, f"wq_{fn}_epilogue")(x, layer), getattr(wq, f"wq_{fn}")(x, layer))
        plain = wq.linear(x, layer)
        assert torch.equal(wq.linear(x, layer, act="none"), plain)
        zero = torch.zeros(160, dtype=torch.float16, device="cuda")
        assert torch.equal(wq.linear(x, layer, bias=zero), plain)
        assert torch.equal(wq.linear(x, layer, act="relu"), torch.relu(plain))
        got = wq.linear(x, layer, residual=plain.clone()).float()
        assert bool(((got - 2 * plain.float()).abs() <= plain.float().abs() * 2.0 ** -9 + 1e-6).all())


@pytest.mark.parametrize("M", [2, 64])
def test_epilogue_ordinary_values(orc, wq, M):
    """Ordinary weights and activations, within the product's own tolerance (SiLU and GELU change a value by at most
    1.13 times the change of their argument)."""
    L = wl.make_layer(2048, 256, 4, 128, wl.ZERO_F16, 8)
    x = wl.make_x(M, 2048, wl.BF16, 4)
    rng = np.random.Generator(np.random.PCG64(1))
    bias, res = wl.to_act_bits(rng.standard_normal(256), wl.BF16), wl.to_act_bits(rng.standard_normal((M, 256)), wl.BF16)
    y64 = oracle_y(orc, x, wl.BF16, L)
    layer = repack_layer(wq, L)
    for act in ACTS:
        y = wq.linear(*(bits_to_tensor(x, torch.bfloat16, "cuda"), layer), bias=bits_to_tensor(bias, torch.bfloat16, "cuda"),
                      act=act, residual=bits_to_tensor(res, torch.bfloat16, "cuda"))
        want = activate(y64 + f64(bias, wl.BF16), act) + f64(res, wl.BF16)
        err = float(np.max(np.abs(tensor_f64(y) - want)))
        _, _, bound = within_tolerance(y64, y64)
        assert err <= 1.13 * bound + 2.0 ** -8 * float(np.max(np.abs(want)))


def test_epilogue_far_values(wq):
    """Activations far below and above zero: no NaN, the limits 0 and v; NaN stays NaN."""
    L = wl.make_layer(256, 16, 4, -1, wl.SYM, 1)
    layer = repack_layer(wq, L)
    x = torch.zeros(3, 256, dtype=torch.float16, device="cuda")
    bias = torch.tensor([-6e4, 6e4, -100, 100, -20, 20, 0, float("nan")] * 2, dtype=torch.float16, device="cuda")
    for act in ACTS:
        y = wq.linear(x, layer, bias=bias, act=act).cpu()
        assert bool(y[:, 7].isnan().all()) and not bool(y[:, :7].isnan().any())
        assert bool((y[:, 1] == bias[1].cpu()).all()) and bool((y[:, 3] == 100).all())
        if act != "none":
            assert bool((y[:, 0] == 0).all()) and float(y[:, 4].abs().max()) < 1e-7


def test_epilogue_in_a_graph(wq):
    """The residual stream added in place, captured and replayed: every replay adds once more."""
    L = wl.make_layer(1024, 64, 4, 128, wl.SYM, 2)
    layer = repack_layer(wq, L)
    for M in (1, 40):
        x = bits_to_tensor(wl.make_x(M, 1024, wl.F16, 3), torch.float16, "cuda") / 64
        y = torch.zeros(M, 64, dtype=torch.float16, device="cuda")
        need = wq.wq_workspace_bytes(M, 64, 1024, 4, False)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        want = torch.zeros_like(y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            wq.linear(x, layer, out=y, ws=ws, residual=y)
        for _ in range(3):
            want = wq.linear(x, layer, residual=want)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
