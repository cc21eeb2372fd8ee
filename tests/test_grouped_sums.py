"""Precision of the grouped products' sums over long reductions, where it shows: on values between
1/2 and 1 every sum is one of like terms, nothing cancels, and an error of the sum, a lost term or a
rounding too early stands out against the result itself.

Tolerance, relative to the result.  A tensor-core step adds 16 products into an fp32 accumulator and
may truncate twice (the aligned products, the sum), at most 2^-23 of the running sum each time.  Over a
piece of P elements the running sum grows in P / 16 equal steps, so the piece is off by at most
2^-22 (P / 32 + 1/2) of itself.  n / P pieces are then added with round to nearest, 2^-24 of a sum that
again grows evenly: 2^-25 (n / P + 1).  fp32 results take pieces of 640 elements: 4.9e-6 and the pieces'
sum.  bf16 weight gradients take pieces of 65536 rows: 4.9e-4 and, up to 2^28 rows, 1.2e-4; below 2^-10
whatever the length, beside the 2^-8 of the result's own rounding."""
import pytest
import torch

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe


def _tol(n, dtype):
    if dtype == BF16:
        return 2.0 ** -8 + 2.0 ** -10
    return 2.0 ** -22 * 20.5 + 2.0 ** -25 * (n / 640 + 1)


def _near(got, ref, n, what):
    rel = ((got.double() - ref).abs() / ref).max().item()
    assert rel <= _tol(n, got.dtype), f"{what}: {rel:.3g} of {_tol(n, got.dtype):.3g}"


def _values(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device="cuda").uniform_(0.5, 1.0, generator=g)


def _offsets(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def _gram(x, dy, rows=1 << 22):
    """x^T dy in float64, some rows at a time."""
    return sum(x[r:r + rows].double().t() @ dy[r:r + rows].double() for r in range(0, len(x), rows))


def test_the_tolerance_sees_what_it_should():
    """A result rounded to bf16, one without its last term and one from a single accumulator (measured:
    1.1e-9 an element) are all refused at the lengths below."""
    g = torch.Generator().manual_seed(0)
    for n in (632, 2880, 16384):
        a, b = (torch.empty((64, n)).uniform_(0.5, 1.0, generator=g).to(BF16).double() for _ in range(2))
        ref = (a * b).sum(1)
        wrong = {"bf16": ref.to(BF16).double(), "a term lost": ref - a[:, -1] * b[:, -1]}
        if n > 5760:
            wrong["one accumulator"] = ref * (1 - 1.1e-9 * n)
        for name, got in wrong.items():
            assert ((got - ref).abs() / ref).max() > 2 * _tol(n, F32), (n, name)


@pytest.mark.gpu
@pytest.mark.parametrize("transpose", [False, True], ids=["product", "transposed"])
@pytest.mark.parametrize("counts", [[1, 3, 0, 2], [100, 128, 70, 1], [300, 256, 0, 511]], ids=["few", "mid", "many"])
@pytest.mark.parametrize("n", [632, 640, 648, 1272, 1280, 1288, 2880, 5760, 16384])
def test_fp32_products(n, counts, transpose):
    K, N = (136, n) if transpose else (n, 136)
    x, W = _values(n, sum(counts), n), _values(n + 1, 4, K, N)
    layer = moe.Moe(4, 64, 64, 1)
    out = layer.grouped_matmul(x, W, _offsets(counts), transpose=transpose, out_dtype=F32)
    assert layer.sync_status() == moe.MOE_OK
    expert = torch.repeat_interleave(torch.arange(4, device="cuda"), torch.tensor(counts, device="cuda"))
    for e in range(4):
        if counts[e]:
            w = W[e].double()
            _near(out[expert == e], x[expert == e].double() @ (w.t() if transpose else w), n, f"expert {e}")


# (experts, segments, columns): tiles enough for a pair each, or few of them that are split over pairs
LONG = {
    "fp32 pieces": (F32, 8, [639, 640, 641, 1279, 1280, 1281, 0, 1919], 264, 520),
    "fp32 pieces, split": (F32, 1, [6401], 64, 72),
    "fp32, long": (F32, 200, [0] * 30 + [131072, 1] + [0] * 168, 64, 72),
    "bf16, one piece": (BF16, 100, [0] * 98 + [65530, 6], 264, 136),
    "bf16 pieces": (BF16, 100, [0] * 94 + [65535, 65536, 65537, 131072, 131073, 5], 264, 136),
    "bf16 pieces, split": (BF16, 1, [65536 * 8 + 1], 64, 72),
    "bf16, 4 million rows": (BF16, 200, [70] * 199 + [1 << 22], 64, 64),
    "bf16, 16 million rows, split": (BF16, 1, [1 << 24], 64, 8),
}


@pytest.mark.gpu
@pytest.mark.parametrize("case", list(LONG), ids=lambda c: c.replace(", ", "-").replace(" ", "-"))
def test_weight_gradients(case):
    dtype, E, counts, K, N = LONG[case]
    x, dy = _values(1, sum(counts), K), _values(2, sum(counts), N)
    o = _offsets(counts)
    layer = moe.Moe(E, 64, 64, 1)
    dW = layer.grouped_wgrad(x, dy, o, out_dtype=dtype)
    assert layer.sync_status() == moe.MOE_OK
    for e in range(E):
        lo, hi = int(o[e]), int(o[e + 1])
        if counts[e] == 0:
            assert (dW[e] == 0).all()
        else:
            _near(dW[e], _gram(x[lo:hi], dy[lo:hi]), counts[e], f"expert {e}")


@pytest.mark.gpu
def test_weight_gradient_of_the_most_rows():
    R = 1 << 28
    x, dy = _values(3, R, 8), _values(4, R, 8)
    layer = moe.Moe(1, 64, 64, 1)
    dW = layer.grouped_wgrad(x, dy, torch.tensor([0, R - 3], dtype=torch.int32, device="cuda"))
    assert layer.sync_status() == moe.MOE_OK
    _near(dW[0], _gram(x[:R - 3], dy[:R - 3], 1 << 25), R - 3, "dW")
