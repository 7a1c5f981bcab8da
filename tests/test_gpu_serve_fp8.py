"""8-bit floating point with block scales on the GPU against the 64-bit oracle: the quantizer's
codes and scales are equal byte for byte, the product lies within its derived error bound."""
import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def g():
    import post_weight_quantization_06_b200 as lib
    return lib


def np64(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    return t.view(torch.uint8).cpu().numpy() if t.is_contiguous() else t.contiguous().view(
        torch.uint8).cpu().numpy()


def values(rows, cols, dtype, seed=0, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen)
    x = x * torch.exp(spread * torch.randn(1, cols, generator=gen) / 3)
    return x.to(DT[dtype]).to(DEV)


# ------------------------------------------------------------------------------------------
# quantizer
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (1, 6144), (3, 129), (128, 128), (130, 257),
                                       (257, 1000), (64, 7), (129, 8), (1000, 384)])
def test_quantize_equals_the_oracle(g, dtype, block_rows, rows, cols):
    X = values(rows, cols, dtype, seed=rows + cols)
    codes, scales = g.fp8_quantize(X, block_rows=block_rows)
    g.gptq_sync_status()
    want, ws = serve.fp8_quantize(np64(X), block_rows)
    assert codes.shape == X.shape and codes.stride(0) % 16 == 0
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(raw(codes), want)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extreme_magnitudes(g, block_rows):
    X = torch.zeros(6, 300)
    X[1, :] = torch.linspace(-1e-44, 1e-44, 300)      # subnormal: the scale stops at 2^-126
    X[2, :] = torch.linspace(-3e38, 3e38, 300)        # its own step overflows: not all finite
    X[3, 5] = 1e-30
    X[4, :] = 448.0
    X[5, :] = -(2.0 ** torch.linspace(-20, 0, 300))   # values that become subnormal codes
    for dt in (torch.float32, torch.bfloat16):
        x = X.to(dt).to(DEV)
        codes, scales = g.fp8_quantize(x, block_rows=block_rows)
        st, info = g.gptq_sync_status(raise_on_error=False)
        assert (st, info) == ((0, 0) if torch.isfinite(x).all() else (g.GPTQ_ERR_NONFINITE, 2))
        want, ws = serve.fp8_quantize(np64(x), block_rows)
        assert np.array_equal(scales.cpu().numpy(), ws)
        # a zero keeps the sign of what it was rounded from on both sides; a NaN has either
        got = raw(codes)
        nan = want & 127 == 127
        assert np.array_equal(np.where(nan, got & 127, got), np.where(nan, want & 127, want))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_the_largest_finite_values(g, block_rows):
    X = torch.tensor([[3.4e38, -3.4e38, 1e38, 1e30] * 40, [1e37, 2e37, -2e36, 0.0] * 40])
    x = X.to(DEV)
    codes, scales = g.fp8_quantize(x, block_rows=block_rows)
    g.gptq_sync_status()
    want, ws = serve.fp8_quantize(np64(x), block_rows)
    assert np.array_equal(scales.cpu().numpy(), ws) and np.array_equal(raw(codes), want)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_reports_what_is_not_finite(g, block_rows, bad):
    X = values(140, 300, "bf16", seed=3)
    X[131, 200] = bad
    codes, scales = g.fp8_quantize(X, block_rows=block_rows)
    st, info = g.gptq_sync_status(raise_on_error=False)
    assert st == g.GPTQ_ERR_NONFINITE and info == 131
    want, ws = serve.fp8_quantize(np64(X), block_rows)
    got = raw(codes)
    assert got[131, 200] & 127 == 127
    got[131, 200] = 127
    assert np.array_equal(got, want) and np.array_equal(scales.cpu().numpy(), ws)
    assert np.isfinite(scales.cpu().numpy()).all()


def test_quantize_a_block_without_a_finite_value(g):
    X = torch.full((2, 130), float("nan"), device=DEV)
    X[0, 129] = 3.0
    codes, scales = g.fp8_quantize(X)
    g.gptq_sync_status(raise_on_error=False)
    want, ws = serve.fp8_quantize(np64(X), 1)
    assert np.array_equal(raw(codes) & 127, want & 127) and np.array_equal(scales.cpu().numpy(), ws)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("offset,pitch", [(0, 264), (1, 259), (4, 300)])
def test_quantize_strided_rows_and_untouched_pitch(g, block_rows, offset, pitch):
    rows, cols = 131, 250
    buf = values(rows + 1, pitch, "bf16", seed=9).reshape(-1)
    X = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    store = torch.full((rows, 256 + offset), 0x5a, dtype=torch.uint8, device=DEV)
    codes = store.view(F8)[:, :cols]
    scales = torch.empty(-(-rows // block_rows), 2, device=DEV)
    g.gptq_fp8_quantize(X, block_rows, codes, scales)
    g.gptq_sync_status()
    want, ws = serve.fp8_quantize(np64(X), block_rows)
    out = store.cpu().numpy()
    assert np.array_equal(out[:, :cols], want) and np.array_equal(scales.cpu().numpy(), ws)
    assert (out[:, cols:] == 0x5a).all()


def test_quantize_empty(g):
    before = g.gptq_launch_count()
    for shape in ((0, 5), (5, 0)):
        codes, scales = g.fp8_quantize(torch.zeros(shape, device=DEV))
        assert codes.shape == shape
    assert g.gptq_launch_count() == before


# ------------------------------------------------------------------------------------------
# product
# ------------------------------------------------------------------------------------------

def operands(g, m, n, k, seed=0):
    A, sA = g.fp8_quantize(values(m, k, "fp32", seed=seed))
    B, sB = g.fp8_quantize(values(n, k, "fp32", seed=seed + 1), block_rows=128)
    return A, sA, B, sB


def judge(Y, A, sA, B, sB, dtype):
    """Each block's 128 products are exact in fp32; their fp32 sum is off by at most 127 roundings
    of at most a step (2^-23, truncating) of the magnitudes; the product of the scales, the
    scaling and the sum over kb blocks and their parts add at most kb + 3 half steps; the output
    one half step of its type."""
    want, mag = serve.fp8_matmul(raw(A), sA.cpu().numpy(), raw(B), sB.cpu().numpy())
    kb = sA.shape[1]
    bound = (127 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * mag
    bound = bound + (np.abs(want) + bound) * torch.finfo(DT[dtype]).eps / 2
    if dtype == "fp16":
        bound = bound + 2.0 ** -25   # half the smallest step
    err = np.abs(np64(Y) - want)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    print(f"worst error {worst:.3f} of the bound")
    assert worst <= 1.0


SHAPES = [(1, 128, 128), (1, 2048, 6144), (1, 1, 16), (2, 130, 17), (7, 200, 1000), (16, 128, 4096),
          (17, 300, 257), (33, 1000, 640), (64, 6144, 256), (65, 129, 129), (127, 257, 511),
          (128, 128, 128), (200, 640, 3000), (256, 256, 256), (300, 513, 130), (777, 1500, 2900),
          (1024, 1024, 1024), (1500, 2050, 400)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_matmul_within_its_bound(g, m, n, k, dtype):
    ops = operands(g, m, n, k, seed=m + n + k)
    Y = g.fp8_matmul(*ops, out_dtype=DT[dtype])
    g.gptq_sync_status()
    judge(Y, *ops, dtype)


def test_matmul_full_size(g):
    """The 2048 x 6144 layer under a long prompt, on sampled rows."""
    m, n, k = 5000, 2048, 6144
    A, sA, B, sB = operands(g, m, n, k)
    Y = g.fp8_matmul(A, sA, B, sB)
    g.gptq_sync_status()
    at = torch.tensor([0, 1, 127, 128, 255, 256, 2500, 4863, 4864, 4991, 4992, 4999], device=DEV)
    sub = A.view(torch.uint8)[at].view(F8)
    judge(Y[at], sub, sA[at], B, sB, "bf16")


def test_matmul_ignores_what_lies_behind_the_columns_and_rows(g):
    m, n, k = 40, 150, 200
    A, sA, B, sB = operands(g, m, n, k)
    pads = []
    for t in (A, B):
        p = torch.full((t.shape[0] + 3, 256), 0x7f, dtype=torch.uint8, device=DEV)   # NaN codes
        p[:t.shape[0], :k] = t.view(torch.uint8)
        pads.append(p.view(F8)[:t.shape[0], :k])
    out = torch.full((m + 1, n + 5), -7.0, device=DEV)
    g.gptq_fp8_matmul(pads[0], sA, pads[1], sB, out[:m, :n])
    g.gptq_sync_status()
    judge(out[:m, :n], A, sA, B, sB, "fp32")
    assert (out[m:] == -7).all() and (out[:, n:] == -7).all()


@pytest.mark.parametrize("m", [5, 300])
def test_matmul_nan_stays_in_its_row_and_column(g, m):
    n, k = 260, 300
    A, sA, B, sB = operands(g, m, n, k)
    A.view(torch.uint8)[3, 290] = 0x7f
    B.view(torch.uint8)[200, 5] = 0xff
    Y = g.fp8_matmul(A, sA, B, sB, out_dtype=torch.float32)
    g.gptq_sync_status()
    nan = torch.isnan(Y)
    want = torch.zeros_like(nan)
    want[3] = True
    want[:, 200] = True
    assert torch.equal(nan, want)


def test_matmul_empty_and_no_columns(g):
    e = torch.empty
    Y = torch.full((3, 4), 5.0, device=DEV)
    g.gptq_fp8_matmul(e(3, 0, device=DEV).to(F8), e(3, 0, device=DEV), e(4, 0, device=DEV).to(F8),
                      e(1, 0, device=DEV), Y)
    g.gptq_sync_status()
    assert (Y == 0).all()
    before = g.gptq_launch_count()
    A, sA, B, sB = operands(g, 4, 4, 32)
    before = g.gptq_launch_count()
    g.gptq_fp8_matmul(A[:0], sA[:0], B, sB, e(0, 4, device=DEV))
    assert g.gptq_launch_count() == before


@pytest.mark.parametrize("m", [1, 48, 700])
def test_matmul_repeats_bit_for_bit_on_streams_and_in_graphs(g, m):
    n, k = 1024, 1100
    a = operands(g, m, n, k, seed=5)
    b = operands(g, m, n, k, seed=50)
    wa, wb = g.fp8_matmul(*a), g.fp8_matmul(*b)
    g.gptq_sync_status()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ya, yb = torch.zeros_like(wa), torch.zeros_like(wb)
    torch.cuda.synchronize()
    for _ in range(5):   # two calls at once
        g.gptq_fp8_matmul(*a, ya, stream=s1)
        g.gptq_fp8_matmul(*b, yb, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(ya, wa) and torch.equal(yb, wb)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for graph, ops, y in ((ga, a, ya), (gb, b, yb)):
        with torch.cuda.graph(graph):
            g.gptq_fp8_matmul(*ops, y)
    ya.zero_()
    yb.zero_()
    for _ in range(3):
        ga.replay()
        gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(ya, wa) and torch.equal(yb, wb)
    g.gptq_sync_status()


def test_a_captured_step_follows_its_inputs(g):
    """Quantize and multiply as one graph: a replay works on what the inputs hold then."""
    m, n, k = 24, 512, 768
    X = values(m, k, "bf16", seed=1)
    _, _, B, sB = operands(g, 1, n, k, seed=2)
    codes, scales = g.fp8_quantize(X)
    Y = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gptq_fp8_quantize(X, 1, codes, scales)
        g.gptq_fp8_matmul(codes, scales, B, sB, Y)
    for seed in (11, 12, 13):
        X.copy_(values(m, k, "bf16", seed=seed))
        graph.replay()
        want = g.fp8_matmul(*g.fp8_quantize(X), B, sB)
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
    g.gptq_sync_status()


@pytest.mark.parametrize("n,dtype", [(2816, "bf16"), (2816, "fp32"), (2801, "bf16"), (2801, "fp16"),
                                     (2802, "bf16"), (2801, "fp32"), (2630, "bf16"), (2624, "fp16")])
def test_matmul_rows_of_any_alignment_at_large_sizes(g, n, dtype):
    """The large-size kernel's stores: whole boxes, ragged last boxes, rows that start between two
    32-bit words. Two sampled row blocks, and every column of them."""
    m, k = 3000, 300
    A, sA, B, sB = operands(g, m, n, k)
    Y = g.fp8_matmul(A, sA, B, sB, out_dtype=DT[dtype])
    g.gptq_sync_status()
    at = torch.cat([torch.arange(0, 40), torch.arange(1270, 1300), torch.arange(2960, 3000)]).to(DEV)
    judge(Y[at], A.view(torch.uint8)[at].view(F8), sA[at], B, sB, dtype)
    assert torch.isfinite(Y).all()


@pytest.mark.parametrize("n,ldy,dtype", [(2630, 2640, "bf16"), (2631, 2632, "fp16"), (2601, 2604, "fp32"),
                                         (2630, 2643, "bf16")])
def test_matmul_into_a_pitched_output_at_large_sizes(g, n, ldy, dtype):
    m, k = 2900, 260
    A, sA, B, sB = operands(g, m, n, k, seed=3)
    out = torch.full((m + 1, ldy), -7.0, device=DEV, dtype=DT[dtype])
    g.gptq_fp8_matmul(A, sA, B, sB, out[:m, :n])
    g.gptq_sync_status()
    at = torch.cat([torch.arange(0, 20), torch.arange(2860, 2900)]).to(DEV)
    judge(out[at, :n], A.view(torch.uint8)[at].view(F8), sA[at], B, sB, dtype)
    assert torch.isfinite(out).all()
    assert (out[m:] == -7).all() and (out[:, n:] == -7).all()


def test_capture_that_forks_and_joins(g):
    """The two operands are quantized on two captured streams and multiplied after the join."""
    m, n, k = 100, 384, 512
    X, W = values(m, k, "bf16", seed=1), values(n, k, "bf16", seed=2)
    A, sA = g.fp8_quantize(X)
    B, sB = g.fp8_quantize(W, block_rows=128)
    Y = torch.zeros(m, n, device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        g.gptq_fp8_quantize(X, 1, A, sA)
        with torch.cuda.stream(side):
            g.gptq_fp8_quantize(W, 128, B, sB)
        main.wait_stream(side)
        g.gptq_fp8_matmul(A, sA, B, sB, Y)
        Y.mul_(2.0)
    for seed in (5, 6):
        X.copy_(values(m, k, "bf16", seed=seed))
        W.copy_(values(n, k, "bf16", seed=seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        a, b = g.fp8_quantize(X), g.fp8_quantize(W, block_rows=128)
        assert torch.equal(Y, 2 * g.fp8_matmul(*a, *b, out_dtype=torch.float32))
    g.gptq_sync_status()


FIRST = """
import torch, post_weight_quantization_06_b200 as g
x = torch.randn(40, 256, device="cuda"); w = torch.randn(300, 256, device="cuda")
at = torch.arange(600, device="cuda") % 300
kv = torch.randn(600, 2, 64, device="cuda", dtype=torch.bfloat16)
c = g.kv_cache(300, 2, 64)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = g.fp8_matmul(*g.fp8_quantize(x), *g.fp8_quantize(w, block_rows=128))
    g.cache_write(c, kv, kv, at)
    k, v = g.cache_read(c, at)
graph.replay()
torch.cuda.synchronize()
want = g.fp8_matmul(*g.fp8_quantize(x), *g.fp8_quantize(w, block_rows=128))
g.cache_write(c, kv, kv, at)
assert torch.equal(y, want) and torch.equal(k, g.cache_read(c, at)[0]) and torch.equal(k, v)
g.gptq_sync_status()
print("ok")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stderr[-2000:]


def judge_columns(Y, A, sA, B, sB, dtype, blocks):
    """`judge` on some blocks of 128 columns."""
    for j in blocks:
        at = slice(128 * j, min(128 * j + 128, B.shape[0]))
        judge(Y[:, at], A, sA, B[at], sB[j:j + 1], dtype)


@pytest.mark.parametrize("m,n,k", [(1, 8192, 8192), (16, 8192, 8192), (20, 8192, 8192), (32, 8064, 8100),
                                   (1, 128, 40000), (25, 300, 30000)])
def test_matmul_few_rows_with_many_blocks_a_cta(g, m, n, k):
    """More blocks of K in a CTA than it has stages, scale slots and accumulators."""
    ops = operands(g, m, n, k, seed=n + k)
    Y = g.fp8_matmul(*ops, out_dtype=torch.float32)
    g.gptq_sync_status()
    last = (n - 1) // 128
    judge_columns(Y, *ops, "fp32", sorted({0, last // 2, last}))


@pytest.mark.parametrize("m,n,k", [(200, 3000, 3000), (40, 128, 20000), (130, 9000, 1700)])
def test_matmul_tiles_with_many_blocks_a_cta(g, m, n, k):
    ops = operands(g, m, n, k, seed=n + k)
    Y = g.fp8_matmul(*ops, out_dtype=torch.float32)
    g.gptq_sync_status()
    last = (n - 1) // 128
    judge_columns(Y, *ops, "fp32", sorted({0, last // 2, last}))


@pytest.mark.parametrize("shift", [0, 1])   # scales that start on 16 bytes, and 4 bytes behind
@pytest.mark.parametrize("k", [640, 900, 1024, 1700])
def test_matmul_large_sizes_with_any_number_of_blocks(g, k, shift):
    m, n = 3000, 2816
    A, sA, B, sB = operands(g, m, n, k, seed=k)
    moved = torch.zeros(sA.numel() + shift, device=DEV)
    moved[shift:] = sA.reshape(-1)
    sA = moved[shift:].view(sA.shape)
    assert sA.data_ptr() % 16 == 4 * shift
    Y = g.fp8_matmul(A, sA, B, sB, out_dtype=torch.float32)
    g.gptq_sync_status()
    # rows of the first tiles of a CTA pair and of its later ones
    at = torch.cat([torch.arange(0, 12), torch.arange(250, 262), torch.arange(2040, 2060),
                    torch.arange(2980, 3000)]).to(DEV)
    judge(Y[at], A.view(torch.uint8)[at].view(F8), sA[at], B, sB, "fp32")
    assert torch.isfinite(Y).all()


def test_matmul_nan_stays_in_its_row_and_column_at_large_sizes(g):
    m, n, k = 3000, 2816, 300
    A, sA, B, sB = operands(g, m, n, k)
    A.view(torch.uint8)[2077, 290] = 0x7f
    B.view(torch.uint8)[1500, 5] = 0xff
    Y = g.fp8_matmul(A, sA, B, sB, out_dtype=torch.float32)
    g.gptq_sync_status()
    want = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    want[2077] = True
    want[:, 1500] = True
    assert torch.equal(torch.isnan(Y), want)


def test_the_product_of_one_token_is_the_nearest_to_its_fp32_sums_each_time(g):
    ops = operands(g, 1, 2048, 6144, seed=4)
    wide = g.fp8_matmul(*ops, out_dtype=torch.float32)
    first = g.fp8_matmul(*ops)
    assert torch.equal(first, wide.to(torch.bfloat16))
    for _ in range(20):
        assert torch.equal(g.fp8_matmul(*ops), first)
    g.gptq_sync_status()
