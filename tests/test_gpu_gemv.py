"""Matrix-vector products with an int4 group-32 matrix (redmoe_gemv) against 64 bits.

Tolerance: products are exact; the sums' error is bounded in plain_ops.gemv_err, and a stored value
adds half a step of its type.
"""

import pytest
import torch

import moe_inputs as mi
import sparse_moe_gemv_b200 as smg
from plain_ops import gemv_err, gemv_rows, store_tol

pytestmark = pytest.mark.gpu


def make(N, K, T, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(31 + seed)
    w, s = mi.quantize_int4g32(torch.randn(N, K, generator=g, device="cuda"))
    return w, s, torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)


def run(w, s, x, out="f32", pad=2):
    N, K, T = w.shape[0], x.shape[1], x.shape[0]
    y = torch.full((T + pad, N), 7.0, device="cuda", dtype=smg.TORCH_DTYPES[out])
    smg.redmoe_gemv(smg.Matrix(w, s, N, K), x, y[:T])
    torch.cuda.synchronize()
    assert bool((y[T:] == 7.0).all())
    return y[:T]


def check(w, s, x, y, rows=None):
    v, m, ms = gemv_rows(w, s, x, rows)
    y = (y if rows is None else y[:, rows]).cpu()
    bad = (y.double() - v).abs() - store_tol(v, gemv_err(m, ms, x.shape[1]), y.dtype)
    assert not y.isnan().any() and float(bad.max()) <= 0, f"{float(bad.max()):.3e} beyond its bound"


@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("N,K,out", [(1, 32, "f32"), (16, 64, "bf16"), (37, 96, "f32"), (512, 2048, "f32"),
                                     (515, 1056, "bf16"), (2048, 512, "bf16"), (100, 4128, "f32")])
def test_sizes(gpu_lib, N, K, T, out):
    w, s, x = make(N, K, T)
    check(w, s, x, run(w, s, x, out))


@pytest.mark.parametrize("N,K,T", [(33, 32768, 32), (16, 65536, 1), (24, 65536, 2), (40, 16384, 13), (9000, 256, 5),
                                   (40000, 128, 1), (40001, 64, 12), (70, 11008, 8), (70, 12000, 7), (90, 5376, 16),
                                   (50, 2560, 31), (4800, 512, 4), (4740, 4096, 8), (1100, 288, 7), (1200, 288, 9),
                                   (600, 7040, 32)])
def test_long_and_wide(gpu_lib, N, K, T):
    w, s, x = make(N, K, T)
    y = run(w, s, x)
    rows = torch.arange(N) if N * K < 2 ** 22 else torch.cat([torch.arange(20), torch.arange(N - 20, N)]).clamp(0, N - 1)
    check(w, s, x, y, rows)
    assert torch.equal(y, run(w, s, x))  # a fixed order of summation


def test_codes_and_columns_land_where_they_belong(gpu_lib):
    """Unit rows of x pick single columns of W: every nibble of every position, exactly."""
    N, K = 48, 160
    g = torch.Generator().manual_seed(4)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    s = torch.tensor([1.0, 0.5, 2.0, 0.25, 4.0]).to(torch.bfloat16).repeat(N, 1).cuda()
    q = torch.stack(((w.cpu() & 15), (w.cpu() >> 4)), dim=-1).reshape(N, K).double() - 8
    W = q * s.cpu().double().repeat_interleave(32, dim=1)
    for T in (1, 2, 8, 13, 32):
        for k0 in range(0, K, T):
            cols = torch.arange(k0, min(K, k0 + T))
            x = torch.zeros(len(cols), K)
            x[torch.arange(len(cols)), cols] = 1.0
            y = run(w, s, x.to(torch.bfloat16).cuda())
            assert torch.equal(y.cpu().double(), W[:, cols].T)


def test_nan_and_infinity_stay_in_their_token(gpu_lib):
    for T in (2, 7):
        for bad in (float("nan"), float("inf")):
            w, s, x = make(64, 256, T)
            want = run(w, s, x).clone()
            x[1, 40] = bad
            y = run(w, s, x)
            assert torch.equal(y[0], want[0]) and bool(y[1].isnan().all()) and (T == 2 or torch.equal(y[2:], want[2:]))


@pytest.mark.parametrize("T", [1, 2, 5])
def test_tokens_of_any_scale(gpu_lib, T):
    """Rows of x from bf16's subnormals to its largest numbers, one of zeros, and one whose elements
    span 100 powers of two: the same bound relative to each row's own sums."""
    w, s, _ = make(50, 512, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    z = torch.randn(T, 512, generator=g, device="cuda")
    for scale in (2.0 ** -128, 1e-30, 1e-3, 3e4, 1e30):
        x = (z * scale).to(torch.bfloat16)
        y = run(w, s, x)
        v, m, ms = gemv_rows(w, s, x)
        # a result below the smallest normal fp32 is held to that number's half step as well
        assert bool(((y.cpu().double() - v).abs() <= store_tol(v, gemv_err(m, ms, 512), torch.float32) + 2.0 ** -149).all())
    x = torch.zeros(T, 512, device="cuda", dtype=torch.bfloat16)
    assert int(run(w, s, x).count_nonzero()) == 0
    x = torch.randn(T, 512, generator=g, device="cuda") * torch.exp2(torch.arange(512, device="cuda") * (100 / 512) - 50)
    x = x.to(torch.bfloat16)
    check(w, s, x, run(w, s, x))
    top = torch.finfo(torch.bfloat16).max
    x = torch.zeros(T, 512, device="cuda", dtype=torch.bfloat16)
    x[:, 5], x[:, 300] = top, -top
    tiny = (s * 0.0 + 2.0 ** -20).to(torch.bfloat16)
    check(w, tiny, x, run(w, tiny, x))


def test_no_rows_streams_and_graph(gpu_lib):
    w, s, x = make(300, 512, 4)
    m = smg.Matrix(w, s, 300, 512)
    smg.redmoe_gemv(m, x[:0], torch.empty(0, 300, device="cuda"))
    want = run(w, s, x)
    y = torch.empty(4, 300, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        smg.redmoe_gemv(m, x, y)
    st.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smg.redmoe_gemv(m, x, y)
    x.copy_(make(300, 512, 4, seed=1)[2])
    y.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check(w, s, x, y)


@pytest.mark.parametrize("T", [1, 5, 13, 32])
def test_calls_that_feed_one_another(gpu_lib, T):
    """A call's kernel may be placed while the one before it ends: a chain of products, each reading what
    the one before wrote and writing what the one before read, equals the same calls one at a time."""
    mats = [smg.Matrix(*make(512, 512, 1, seed=i)[:2], 512, 512) for i in range(6)]
    x = make(512, 512, T, seed=9)[2] * 0.05
    buf = [x.clone(), torch.empty_like(x)]
    want = x
    for i in range(60):
        y = torch.empty_like(x)
        smg.redmoe_gemv(mats[i % 6], want, y)
        torch.cuda.synchronize()
        want = (y.float() * 2.0 ** -5).to(torch.bfloat16)  # about what 512 products grow by: exact
    scaled = [smg.Matrix(m.w, m.s * 2.0 ** -5, 512, 512) for m in mats]

    def chain():
        for i in range(60):
            smg.redmoe_gemv(scaled[i % 6], buf[i % 2], buf[1 - i % 2])

    chain()
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and float(want.abs().max()) > 0 and torch.equal(buf[0], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    buf[0].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf[0], want)


def test_offsets_beyond_32_bits(gpu_lib):
    """More than 2^31 bytes of packed weights."""
    N, K = 140001, 32768
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w = torch.empty(N, K // 2, device="cuda", dtype=torch.uint8).random_(0, 256, generator=g)
    s = torch.rand(N, K // 32, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(3, K, generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([0, 65535, 131071, 131072, 140000])
    check(w[rows.cuda()], s[rows.cuda()], x, run(w, s, x)[:, rows.cuda()])


def test_binding_refusals_on_the_device(gpu_lib):
    w, s, x = make(64, 128, 2)
    m = smg.Matrix(w, s, 64, 128)
    y = torch.empty(2, 64, device="cuda")
    for bx, by in ((x[:, :64], y), (x, y[:, :32]), (x.half(), y), (x, y.half()), (x.cpu(), y), (x, y[:1])):
        with pytest.raises(ValueError):
            smg.redmoe_gemv(m, bx, by)
    with pytest.raises(smg.RedmoeError, match="UNSUPPORTED"):
        smg.redmoe_gemv(m, x.float(), y)
    with pytest.raises(smg.RedmoeError, match="UNSUPPORTED"):
        smg.redmoe_gemv(m, torch.zeros(33, 128, device="cuda", dtype=torch.bfloat16), torch.empty(33, 64, device="cuda"))
    with pytest.raises(ValueError):
        smg.Matrix(w, s[:, :2], 64, 128)
