"""The INT8 product of several tokens and its activations' quantiser, against
plain 64-bit forms: every code equal, products inside a derived bound."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import serving_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _check_codes(x, label):
    say(f"[quantize tokens] {label}")
    q, s = binding.quantize_tokens_q8(x)
    torch.cuda.synchronize()
    want_q, want_s = ref.quantize_tokens(x.cpu().double().numpy())
    assert np.array_equal(s.cpu().double().numpy(), want_s, equal_nan=True), label
    assert np.array_equal(q.cpu().double().numpy(), want_q), label
    return q, s


# 512 and 1024: rows of one wave; 4096, 8192, 16384: the register-held limits;
# 20000: read twice; 1, 7, 4100 + odd: element-wise
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N", [1, 7, 8, 511, 512, 1024, 1032, 4096, 4104, 4099, 8192, 8200, 16384, 16392, 20000])
def test_codes_and_scales(gpu, dtype, N):
    g = torch.Generator().manual_seed(N)
    for T in (1, 5):
        x = (torch.randn((T, N), generator=g) * 3).to(dtype)
        _check_codes(x.cuda(), f"{T}x{N} {dtype}")


def test_ties_and_borders(gpu):
    # absmax 127 makes the scale 1: every half is a tie; neighbours of ties in
    # binary32 lie one place beside them
    halves = np.arange(-126.5, 127, 1.0, dtype=np.float32)
    x = np.concatenate([[127.0], halves, np.nextafter(halves, np.float32(-200)), np.nextafter(halves, np.float32(200))])
    _check_codes(torch.from_numpy(x.astype(np.float32))[None].cuda(), "ties, scale 1")
    # the same quotients on scales whose products with the codes are inexact
    rng = np.random.default_rng(0)
    rows = []
    for top in rng.uniform(1e-3, 1e3, 64).astype(np.float32):
        s = np.float32(top / np.float32(127))
        k = rng.integers(-127, 127, 255)
        near = ((k + 0.5) * np.float64(s)).astype(np.float32)
        near = np.where(rng.random(255) < 0.5, np.nextafter(near, np.float32(0)), near)
        rows.append(np.concatenate([[top], near]))
    x = np.array(rows, np.float32)
    x = np.clip(x, -x[:, :1], x[:, :1])
    _check_codes(torch.from_numpy(x).cuda(), "ties, any scale")


def test_extreme_rows(gpu):
    x = torch.zeros((9, 64))
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = torch.linspace(-3e38, 3e38, 64)
    x[4] = torch.arange(64) * 2.0 ** -149          # codes of subnormal scales, or of none
    x[5] = torch.arange(64) * 3 * 2.0 ** -149      # the scale rounds: the top code is clipped
    x[6] = torch.arange(64) * 2.0 ** -127
    x[7, 0] = -0.0
    x[8] = -1e-30
    _, s = _check_codes(x.cuda(), "extreme rows")
    assert torch.isnan(s[1]) and torch.isnan(s[2]) and s[0] == 0 and s[7] == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strided_and_unaligned_rows(gpu, dtype):
    g = torch.Generator().manual_seed(5)
    wide = (torch.randn((6, 3 * 520 + 1), generator=g)).to(dtype).cuda()
    _check_codes(wide[:, 520:1040], f"a part of wider rows, {dtype}")     # rows 1561 elements apart: element-wise
    wide = (torch.randn((6, 3 * 520), generator=g)).to(dtype).cuda()
    _check_codes(wide[:, 520:1040], f"a part of wider rows, aligned, {dtype}")
    _check_codes(wide[:, 1:513], f"from an odd element, {dtype}")


def test_empty(gpu):
    q, s = binding.quantize_tokens_q8(torch.empty((0, 64), device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)
    q, s = binding.quantize_tokens_q8(torch.empty((3, 0), device="cuda"))
    torch.cuda.synchronize()
    assert q.shape == (3, 0) and torch.all(s == 0)


# ---------------------------------------------------------------- product
def _operands(T, M, N, seed, low=-127):
    rng = np.random.default_rng(seed)
    return (rng.integers(low, 128, (M, N), dtype=np.int8), rng.uniform(1e-4, 2e-3, M).astype(np.float16),
            rng.integers(low, 128, (T, N), dtype=np.int8), rng.uniform(1e-3, 0.05, T).astype(np.float32))


def _check_product(A, scale, x, xs, dtype, label):
    say(f"[gemm q8] {label}")
    y = binding.gemm_q8(*(torch.from_numpy(t).cuda() for t in (A, scale, x, xs)), out_dtype=dtype)
    torch.cuda.synchronize()
    want = ref.product(A, scale, x, xs)
    off = np.abs(y.cpu().double().numpy() - want)
    assert y.dtype == dtype and y.shape == want.shape
    assert np.all(off <= ref.product_bound(want, dtype)), (label, np.max(off - ref.product_bound(want, dtype)))
    return y


TOKENS = [1, 2, 3, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257, 300, 513]


@pytest.mark.parametrize("T", TOKENS)
def test_products_by_tokens(gpu, T):
    for M, N in ((256, 512), (300, 1040), (64, 4096)):
        _check_product(*_operands(T, M, N, T), torch.float16, f"T={T} M={M} N={N}")


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 129, 255, 257, 400, 1000])
def test_products_by_outputs(gpu, M):
    for T, N in ((1, 512), (20, 256), (130, 128), (260, 64)):
        _check_product(*_operands(T, M, N, M), torch.float32, f"T={T} M={M} N={N}")


# multiples of 16 take the bandwidth path, others do not
@pytest.mark.parametrize("N", [0, 1, 15, 16, 17, 31, 32, 48, 63, 64, 80, 100, 112, 127, 128, 129, 144, 240, 256, 272, 384,
                               500, 1000, 1008, 2064, 4095])
def test_products_by_inner_size(gpu, N):
    for T, M in ((1, 40), (33, 70), (150, 200), (300, 260)):
        for dtype in TYPES:
            _check_product(*_operands(T, M, N, N), dtype, f"T={T} M={M} N={N} {dtype}")


def test_random_shapes(gpu):
    rng = np.random.default_rng(7)
    for i in range(60):
        T, M, N = (int(np.exp(rng.uniform(0, np.log(top)))) for top in (1500, 1500, 4000))
        if i % 3:
            N = -(-N // 16) * 16
        _check_product(*_operands(T, M, N, i), TYPES[i % 3], f"random {i}: T={T} M={M} N={N}")


def test_largest_sums_stay_whole(gpu):
    # all -128: each product 2^14, the sum 131071 * 2^14 just below 2^31; and
    # the most negative one
    for T, M in ((1, 5), (3, 65), (70, 70), (130, 260)):
        for N in (131071, 131056):
            A, x = np.full((M, N), -128, np.int8), np.full((T, N), -128, np.int8)
            A[0] = 127
            _check_product(A, np.ones(M, np.float16), x, np.ones(T, np.float32), torch.float32, f"T={T} N={N} of -128")


def test_unaligned_operands(gpu):
    for T in (1, 20, 100, 300):
        A, s, x, xs = _operands(T, 130, 256, 3)
        a = torch.zeros(130 * 256 + 1, dtype=torch.int8, device="cuda")
        a[1:] = torch.from_numpy(A).cuda().ravel()
        b = torch.zeros(T * 256 + 3, dtype=torch.int8, device="cuda")
        b[3:] = torch.from_numpy(x).cuda().ravel()
        say(f"[gemm q8] unaligned, T={T}")
        y = binding.gemm_q8(a[1:].view(130, 256), torch.from_numpy(s).cuda(), b[3:].view(T, 256),
                            torch.from_numpy(xs).cuda(), out_dtype=torch.float32)
        want = ref.product(A, s, x, xs)
        assert np.all(np.abs(y.cpu().double().numpy() - want) <= ref.product_bound(want, torch.float32))


def test_scales_of_nan_zero_and_infinity(gpu):
    A, s, x, xs = _operands(4, 70, 128, 9)
    xs[1], xs[2] = np.nan, 0.0
    s[3] = 0.0
    y = binding.gemm_q8(*(torch.from_numpy(t).cuda() for t in (A, s, x, xs)), out_dtype=torch.float32).cpu()
    assert torch.all(torch.isnan(y[1])) and torch.all(y[2] == 0) and torch.all(y[[0, 3], 3] == 0)
    assert torch.all(torch.isfinite(y[[0, 2, 3]]))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_nothing_outside_y_is_written(gpu, T):
    A, s, x, xs = (torch.from_numpy(t).cuda() for t in _operands(T, 97, 256, 4))
    for dtype in TYPES:
        buf = torch.full((T * 97 + 64,), 7.0, dtype=dtype, device="cuda")
        y = buf[32: 32 + T * 97].view(T, 97)
        say(f"[gemm q8] guards, T={T} {dtype}")
        binding.gemm_q8(A, s, x, xs, out=y)
        assert torch.all(buf[:32] == 7) and torch.all(buf[32 + T * 97:] == 7)
        assert torch.equal(y, binding.gemm_q8(A, s, x, xs, out_dtype=dtype))


def test_one_token_agrees_with_gemv_q8(gpu):
    # the same weights: on activations that binary16 holds exactly, both give the same sums
    A, s, x, _ = _operands(1, 512, 1024, 6)
    d = [torch.from_numpy(t).cuda() for t in (A, s)]
    y = binding.gemm_q8(*d, torch.from_numpy(x).cuda(), torch.ones(1, device="cuda"), out_dtype=torch.float32)[0]
    z = binding.gemv_q8(*d, torch.from_numpy(x[0].astype(np.float16)).cuda())
    assert torch.allclose(y, z, rtol=1e-3, atol=1e-3 * float(y.abs().max()))


def test_linear_layer_against_its_own_quantisation(gpu):
    # quantise and multiply, as a layer does: the error is that of the codes
    g = torch.Generator().manual_seed(11)
    x = torch.randn((37, 1024), generator=g).to(torch.bfloat16)
    W = torch.randn((200, 1024), generator=g)
    A, s, _ = binding.quantize_q8(W.cuda())
    q, t = binding.quantize_tokens_q8(x.cuda())
    y = binding.gemm_q8(A, s, q, t, out_dtype=torch.float32).cpu().double()
    wd, xd = A.cpu().double() * s.cpu().double()[:, None], x.double()
    # |x - q t| <= t / 2 in each of the summed values
    bound = 0.5 * t.cpu().double()[:, None] * wd.abs().sum(1)[None] * (1 + 1e-6) + 1e-6
    assert torch.all((y - xd @ wd.T).abs() <= bound + 4 * ref.U32 * (xd.abs() @ wd.abs().T))


def test_refusals(gpu):
    A, s, x, xs = (torch.from_numpy(t).cuda() for t in _operands(4, 32, 64, 1))
    with pytest.raises(TypeError):
        binding.gemm_q8(A.to(torch.uint8), s, x, xs)
    with pytest.raises(ValueError):
        binding.gemm_q8(A, s[:-1], x, xs)
    with pytest.raises(ValueError):
        binding.gemm_q8(A, s, x[:, :-16], xs)
    with pytest.raises(ValueError):
        binding.gemm_q8(A, s, x, xs[:-1])
    with pytest.raises(TypeError):
        binding.gemm_q8(A, s, x, xs.double())
    with pytest.raises(TypeError):
        binding.gemm_q8(A, s, x, xs, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        binding.quantize_tokens_q8(torch.zeros((2, 8), dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        binding.quantize_tokens_q8(torch.zeros((8, 4), device="cuda").t())
    with pytest.raises(ValueError):
        binding.quantize_tokens_q8(torch.zeros((8, 4)))
    big = torch.zeros((1, 131072), dtype=torch.int8, device="cuda")
    with pytest.raises(binding.GemvError) as e:
        binding.gemm_q8(big, torch.ones(1, dtype=torch.float16, device="cuda"), big, torch.ones(1, device="cuda"))
    assert e.value.status == 2


def test_large_tiles_whole_and_halved(gpu):
    # tiles of 256 x 256: fewer than the CUs, whole rounds of them, and rounds
    # whose rest is done in halves, one of which may lie past the last output
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 256 * 16
    for tiles_m, short in ((cus * 3 // 4 // 16 + 1, 100), (cus // 16, 0), (cus // 16 + 2, 0), (cus // 16 + 3, 200),
                           (cus // 16 + 9, 128)):
        M, N = tiles_m * 256 - short, 208
        A, s, x, xs = _operands(rows - 7, M, N, tiles_m)
        _check_product(A, s, x, xs, torch.float16, f"{rows - 7}x{M}x{N}")


def test_few_tokens_at_every_tiling(gpu):
    # outputs and tokens such that each tile size is the cheapest once, with
    # columns that end inside a stage
    for T, M, N in ((1, 300, 1040), (5, 4096, 528), (16, 9000, 528), (20, 4000, 272), (32, 9000, 272), (30, 20000, 144),
                    (60, 4000, 528), (64, 20000, 144), (128, 4000, 400), (120, 14336, 144), (300, 8192, 144)):
        _check_product(*_operands(T, M, N, T), torch.bfloat16, f"T={T} M={M} N={N}")
