"""dsa_rms_norm against its definition in 64 bits.

Tolerances, with u the half step of the 16-bit type: z is one fp32 addition
(2^-24); the squares' sum of at most 32 of a thread, 5 + 5 shuffle levels, the
mean and eps is off by at most 48 * 2^-24 (all terms positive), half of that
after the root; root, division, two products and z: 5 more.  So y is within 30 *
2^-24 of itself, and out within u more (fp16: 2^-25 absolute where it is
subnormal).  An e4m3 code is within half a step of y * 2^-e."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
EPS = 1e-6
R = 30 * 2.0 ** -24  # relative error of y in fp32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def inputs(T, N, dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, N, generator=g, device="cuda") * scale).to(dtype)
    res = (torch.randn(T, N, generator=g, device="cuda") * 3 * scale).to(dtype)
    gamma = torch.rand(N, generator=g, device="cuda") * 2 - 0.5
    return x, res, gamma


def definition(x, res, gamma):
    z = x.double() if res is None else x.double() + res.double()
    return z, z / (z.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.double()


def tiny(dtype):
    return 2.0 ** -25 if dtype == FP else 2.0 ** -134


def check16(out, y):
    u = torch.finfo(out.dtype).eps / 2
    assert ((out.double() - y).abs() <= y.abs() * (u * (1 + R) + R) + tiny(out.dtype)).all()


def check_residual(got, z):
    u = torch.finfo(got.dtype).eps / 2
    assert ((got.double() - z).abs() <= z.abs() * (u + 2.0 ** -23) + tiny(got.dtype)).all()


def check8(codes, scales, y, group):
    T, N = y.shape
    if scales.dtype != torch.float32:
        scales = torch.exp2(scales.view(torch.uint8).double() - 127)
    scales = scales.double()
    groups = -(-N // group)
    assert scales.shape == (T, groups) and codes.shape == y.shape
    wide = torch.zeros(T, groups * group, dtype=torch.float64, device="cuda")
    wide[:, :N] = y
    amax = wide.view(T, groups, group).abs().amax(-1).clamp(min=1e-4)
    low, high = (torch.exp2(torch.ceil(torch.log2(amax * f / 448))) for f in (1 - 2 * R, 1 + 2 * R))
    assert ((scales == low) | (scales == high)).all()  # two where y in fp32 may pass a border
    x = wide / scales.repeat_interleave(group, 1)
    got = torch.zeros_like(wide)
    got[:, :N] = codes.view(torch.float8_e4m3fn).double()
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    assert ((got - x).abs() <= step / 2 * (1 + 2.0 ** -20) + x.abs() * 2 * R).all()


SIZES = [(1, 8), (1, 7168), (2, 32768), (3, 24), (5, 264), (64, 4096), (305, 1000), (304, 2048),
         (1000, 136), (700, 5120), (4097, 64), (310, 8200), (306, 32768), (400, 16384), (333, 32)]


@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("residual", [True, False])
def test_16_bits(T, N, dtype, residual):
    import prep_token_gb300 as dp
    x, res, gamma = inputs(T, N, dtype, T + N)
    z, y = definition(x, res if residual else None, gamma)
    if residual:
        out, r = dp.dsa_rms_norm(x, gamma, EPS, residual=res)
        check_residual(r, z)
    else:
        out = dp.dsa_rms_norm(x, gamma, EPS)
    check16(out, y)


@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.float8_e8m0fnu])
def test_8_bits(T, N, group, scale_dtype):
    import prep_token_gb300 as dp
    dtype = BF if (T + N) % 3 else FP
    x, res, gamma = inputs(T, N, dtype, T * 7 + N)
    z, y = definition(x, res, gamma)
    codes, scales, r = dp.dsa_rms_norm_fp8(x, gamma, EPS, residual=res, group=group,
                                           scale_dtype=scale_dtype)
    assert scales.dtype == scale_dtype
    check8(codes, scales, y, group)
    check_residual(r, z)


@pytest.mark.parametrize("T,N", [(3, 7168), (500, 7168), (900, 96)])
def test_both_outputs_strided_and_in_place(T, N):
    import prep_token_gb300 as dp
    wide, res, gamma = inputs(T, N + 40, BF, 3)
    x, res = wide[:, 16:16 + N], res[:, :N]
    gamma = gamma[:N].contiguous()
    z, y = definition(x, res, gamma)
    outside = wide[:, 16 + N:].clone()
    codes = torch.full((T + 2, N + 8), 0x7f, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 1, -(-N // 32) + 3), -1.0, device="cuda")
    got = dp.dsa_rms_norm_fp8(x, gamma, EPS, residual=res, group=32, out=x, residual_out=res,
                              codes=codes[:, :N], scales=scales[:, :-3])
    check8(codes[:T, :N], scales[:T, :-3], y, 32)
    check16(x, y)
    check_residual(res, z)
    assert got[2].data_ptr() == res.data_ptr()
    assert torch.equal(wide[:, 16 + N:], outside)
    assert (codes[T:] == 0x7f).all() and (codes[:, N:] == 0x7f).all()
    assert (scales[T:] == -1).all() and (scales[:, -3:] == -1).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_out_of_the_ordinary(dtype):
    """Rows of zeros, of one value, of the type's smallest and large values; a NaN stays in its row."""
    import prep_token_gb300 as dp
    x, _, gamma = inputs(8, 512, dtype, 5)
    x[0] = 0
    x[1] = 0
    x[1, 300] = 1
    x[2] = torch.finfo(dtype).tiny
    x[3] *= 1e4
    x[4, 17] = math.nan
    x[5] = torch.finfo(dtype).max if dtype == FP else 1e17
    x[6, 511] = 3e4
    rows = [0, 1, 2, 3, 5, 6, 7]
    _, y = definition(x, None, gamma)
    out = dp.dsa_rms_norm(x, gamma, EPS)
    check16(out[rows], y[rows])
    assert torch.isnan(out[4]).all()
    codes, scales = dp.dsa_rms_norm_fp8(x, gamma, EPS)
    check8(codes[rows], scales[rows], y[rows], 128)
    assert (codes[0].view(torch.uint8) & 0x7f == 0).all() and (scales[0] == 2.0 ** -22).all()


def test_amax_at_each_border():
    """Values that are the codes' own at every exponent: amax 448 * 2^e takes e, the next one e + 1."""
    import prep_token_gb300 as dp
    # every value is the root mean square, all of it powers of two: y = gamma exactly
    x = torch.full((1, 4096), 2.0 ** 12, device="cuda", dtype=BF)
    e = torch.arange(-16, 16, device="cuda")
    gamma = (448 * torch.exp2(e.float())).repeat_interleave(128)
    codes, scales = dp.dsa_rms_norm_fp8(x, gamma, 1e-30)
    assert torch.equal(scales[0], torch.exp2(e.float())) and (codes.float() == 448).all()
    above = torch.nextafter(gamma, torch.full_like(gamma, math.inf))
    codes, scales = dp.dsa_rms_norm_fp8(x, above, 1e-30)
    assert torch.equal(scales[0], torch.exp2(e.float() + 1)) and (codes.float() == 224).all()


def test_captured_and_on_another_stream():
    import prep_token_gb300 as dp
    x, res, gamma = inputs(200, 7168, BF, 9)
    out, r = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    dp.dsa_rms_norm(x, gamma, EPS, residual=res, out=out, residual_out=r, stream=side)
    side.synchronize()
    want = definition(x, res, gamma)
    check16(out, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.dsa_rms_norm(x, gamma, EPS, residual=res, out=out, residual_out=r, pdl=True)
        codes, scales = dp.dsa_rms_norm_fp8(out, gamma, EPS, pdl=True)  # reads what the first wrote
    x.copy_(inputs(200, 7168, BF, 10)[0])
    graph.replay()
    torch.cuda.synchronize()
    z, y = definition(x, res, gamma)
    check16(out, y)
    check_residual(r, z)
    check8(codes, scales, definition(out, None, gamma)[1], 128)


def test_same_results_again():
    import prep_token_gb300 as dp
    x, res, gamma = inputs(777, 5120, FP, 11)
    first = dp.dsa_rms_norm_fp8(x, gamma, EPS, residual=res)
    for _ in range(3):
        again = dp.dsa_rms_norm_fp8(x, gamma, EPS, residual=res)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, again))


def test_empty():
    import prep_token_gb300 as dp
    x, res, gamma = inputs(0, 64, BF)
    assert dp.dsa_rms_norm(x, gamma, EPS).shape == (0, 64)
    assert dp.dsa_rms_norm_fp8(x, gamma, EPS)[1].shape == (0, 1)
