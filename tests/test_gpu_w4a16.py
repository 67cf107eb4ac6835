"""Products of a few rows with 4-bit weights against 64 bits.

Tolerance, with S = sum |x q| s over a row's products, which are exact: a step of 128 products is added up by the tensor
core in 8 instructions (24 for fp32 rows, in three parts), each of which may lose 2^-23 of what the step holds; the
steps of a warp, and the warps, are added in fp32, each addition and each scaling 2^-24 of S at most.  Then the one
rounding to the output type."""
import pytest
import torch

import paged_ref
import prefix_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def layer(N, K, grouped, seed):
    g = gen(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.exp(torch.randn(N, K // 128 if grouped else 1, generator=g)) * 0.01
    return codes.to(DEV), (scales if grouped else scales[:, 0]).contiguous().to(DEV)


def check(x, codes, scales, out_dtype=None, **kw):
    got = rq.w4a16_gemm(x, codes, scales, out_dtype=out_dtype, **kw)
    dtype = out_dtype or x.dtype
    assert got.dtype == dtype and got.shape == (x.shape[0], codes.shape[0]) and got.is_contiguous()
    w = ref.weights(codes, scales)
    want, S = x.double() @ w.T, x.double().abs() @ w.abs().T
    eps = (3 if x.dtype == torch.float32 else 1) * 2.0**-20 + (x.shape[1] / 128 + 16) * 2.0**-24
    bound = eps * S + paged_ref.UNIT[dtype] * want.abs() * 1.01 + (2.0**-25 if dtype == torch.float16 else 1e-44)
    err = (got.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 16, 128), (1, 17, 256), (2, 100, 384), (3, 4101, 1024), (5, 15, 2048),
                                   (7, 33, 14336), (8, 1000, 4096), (9, 200, 1152), (16, 129, 4096), (17, 64, 512),
                                   (31, 50, 1408), (33, 70, 256), (61, 1030, 4096), (64, 256, 8192), (1, 2048, 28672),
                                   (2, 5000, 16384), (8, 30, 65536), (13, 3000, 8192), (16, 5001, 8192), (24, 700, 28672),
                                   (3, 20, 262144), (6, 40000, 128), (29, 9000, 1024)])
def test_shapes(dtype, grouped, M, N, K):
    codes, scales = layer(N, K, grouped, M + N)
    check(randn(M, K, seed=K + M, dtype=dtype).to(DEV), codes, scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 6, 40])
def test_output_types(dtype, out_dtype, M):
    codes, scales = layer(130, 640, True, 3)
    check(randn(M, 640, seed=4, dtype=dtype).to(DEV), codes, scales, out_dtype)


@pytest.mark.parametrize("M", range(1, 65))
def test_every_number_of_rows(M):
    codes, scales = layer(300, 1280, True, 5)
    got = check(randn(M, 1280, seed=6, dtype=torch.bfloat16).to(DEV), codes, scales)
    assert got.shape[0] == M


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 8, 50])
def test_exact_sums(dtype, M):
    """Whole numbers below 2^24 come out exactly: all 16 codes against rows of small whole numbers, a scale of one."""
    K, N = 512, 160
    g = gen(7)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).to(DEV)
    x = torch.randint(-100, 101, (M, K), generator=g).to(dtype).to(DEV)
    scales = torch.ones(N, K // 128, device=DEV)
    got = rq.w4a16_gemm(x, codes, scales, out_dtype=torch.float32)
    assert torch.equal(got.double(), x.double() @ ref.weights(codes, scales).T)
    assert torch.equal(got, rq.w4a16_gemm(x, codes, scales[:, 0].contiguous(), out_dtype=torch.float32))
    # one code at a time: which one goes with which element
    eye = torch.eye(K, device=DEV)[:min(M * 8, K)].to(dtype)
    for a in range(0, eye.shape[0], M):
        assert torch.equal(rq.w4a16_gemm(eye[a:a + M], codes, scales, out_dtype=torch.float32).double(),
                           ref.weights(codes, scales).T[a:a + M])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [2, 20])
def test_magnitudes(dtype, M):
    """Rows far apart in size, elements far apart in a row, scales far apart, rows and scales of zero."""
    K, N = 1024, 70
    codes, scales = layer(N, K, True, 8)
    scales *= torch.exp2(20 * torch.rand(N, K // 128, generator=gen(9)) - 10).to(DEV)
    scales[3] = 0.0
    x = randn(M, K, seed=10)
    x[:, 5] *= 300.0
    if dtype == torch.float16:
        x *= torch.exp2(torch.linspace(-8, 3, M))[:, None]
    else:
        x *= torch.exp2(torch.linspace(-60, 40, M))[:, None]
    x[1] = 0.0
    got = check(x.to(dtype).to(DEV), codes, scales, torch.float32)
    assert (got[:, 3] == 0).all() and (got[1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [2, 20])
def test_ends_of_the_range(dtype, M):
    """Rows near the ends of fp32's range, in one step and in another: what fits the output is right."""
    K, N = 512, 40
    codes, scales = layer(N, K, True, 19)
    scales = torch.full_like(scales, 2.0**-20)
    x = randn(M, K, seed=20)
    x /= x.abs().amax()
    x[:, :128] *= 3e38
    x[:, 128:256] *= 1e-30
    x[1] *= 1e-25
    check(x.to(dtype).to(DEV), codes, scales, torch.float32)
    check((x[:, 128:256] * 1e-8).to(dtype).to(DEV), codes[:, :64].contiguous(), torch.ones(N, 1, device=DEV), torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [3, 30])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_are_not_finite(dtype, M, bad):
    """A NaN or an infinity reaches its own row alone, and all of that."""
    codes, scales = layer(90, 512, True, 11)
    x = randn(M, 512, seed=12, dtype=dtype)
    clean = rq.w4a16_gemm(x.to(DEV), codes, scales)
    x[1, 77] = bad
    got = rq.w4a16_gemm(x.to(DEV), codes, scales)
    keep = torch.arange(M) != 1
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[1]).any()


@pytest.mark.parametrize("M", [1, 4, 33])
def test_strides_outputs_streams_and_repeats(M):
    K, N = 768, 203
    codes, scales = layer(N, K, True, 13)
    rows = randn(M, 2 * K, seed=14, dtype=torch.bfloat16).to(DEV)
    x = rows[:, K:]                                             # rows 2 K apart
    want = check(x.contiguous(), codes, scales)
    assert torch.equal(check(x, codes, scales), want)
    if M > 1:
        assert torch.equal(rq.w4a16_gemm(rows[:1, K:].expand(M, K), codes, scales), want[:1].expand(M, N))
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert rq.w4a16_gemm(x, codes, scales, out=out) is out and torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rq.w4a16_gemm(x, codes, scales, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rq.w4a16_gemm(x, codes, scales)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert rq.w4a16_gemm(x[:0], codes, scales).shape == (0, N)
    assert rq.w4a16_gemm(x, codes[:0], scales[:0]).shape == (M, 0)


def test_weights_past_32_bits():
    """Codes, and results, at byte offsets that pass 2^32."""
    N, K = 140000, 65536
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.ones(N, device=DEV)
    g = gen(21)
    for n in (0, 1, 65536, 131071, 131072, 139999):
        codes[n] = torch.randint(0, 256, (K // 2,), generator=g, dtype=torch.uint8).to(DEV)
    at = torch.tensor([0, 1, 2, 65536, 131071, 131072, 139998, 139999], device=DEV)
    x = torch.randint(-3, 4, (2, K), generator=g).to(torch.bfloat16).to(DEV)
    got = rq.w4a16_gemm(x, codes, scales, out_dtype=torch.float32)
    assert torch.equal(got[:, at].double(), x.double() @ ref.weights(codes[at], scales[at]).T)


def test_nothing_is_written_beside_the_output():
    for M, N in ((1, 17), (5, 33), (40, 131)):
        codes, scales = layer(N, 256, True, 15)
        pad = torch.full((M * N + 64,), 5.0, dtype=torch.float16, device=DEV)
        x = randn(M, 256, seed=16, dtype=torch.float16).to(DEV)
        rq.w4a16_gemm(x, codes, scales, out=pad[:M * N].view(M, N))
        assert (pad[M * N:] == 5.0).all()


@pytest.mark.parametrize("M", [1, 12, 60])
def test_rotated_layer(M):
    """The layer a user builds: weights folded with their scales, rows rotated, y close to the unrotated product."""
    K, N = 2048, 320
    x, wt = randn(M, K, seed=17).to(DEV), (randn(N, K, seed=18) * 0.02).to(DEV)
    w, s = rq.fwht_quant(wt, SEED, rq.RQ_SIGNS_FIRST | rq.RQ_GROUP_SCALES)
    rows = rq.fwht_quant(x, SEED, want_y=True)[2]
    got = check(rows, w, s)
    want = x.double() @ wt.double().T
    # 4-bit weights with a scale for each 128: half a step of about 2.7 sigma / 7, uniform: 11% of the weights
    assert float((got.double() - want).norm() / want.norm()) < 0.15
