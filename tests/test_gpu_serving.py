"""The 8-bit serving entries on the GPU against their float64 definitions."""
import numpy as np
import pytest
import torch

import post_int4_weight_gptq_b200 as piq
from oracle import serving as S

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def worst(err, tol):
    """The largest err / tol (0 where both are 0); NaN has to be expected: it counts as inf."""
    r = np.divide(err, tol, out=np.zeros_like(err), where=err != 0)
    return float(np.nan_to_num(r, nan=np.inf).max(initial=0.0))


def rand(rng, shape, dtype, std=1.0):
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).cuda().to(dtype)


def f32(t):
    return t.detach().float().cpu().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------- linear
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (7, 72), (33, 1024), (5, 1032), (3, 4104),
                                       (2, 16392), (2, 40000)])
def test_quantize_rows_is_the_definition(dtype, rows, cols):
    rng = np.random.default_rng(rows * cols)
    x = rand(rng, (rows, cols), dtype)
    x[0, cols // 2] = 30.0
    if rows > 2:
        x[1] = 0
        x[2, 1] = float("inf")
        x[2, 5] = float("nan")
    codes, scales = piq.int8_quantize_rows(x)
    c, s = S.quantize_rows_ref(f32(x))
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)


def test_quantize_rows_extremes():
    x = torch.zeros(6, 64, device="cuda")
    x[0, 3] = 1e-37          # its scale is a subnormal number: 0
    x[1, 3] = 3e-36          # the smallest scales that are kept
    x[2, :2] = torch.tensor([3.4e38, -1e38])
    x[3, 0] = -float("inf")
    x[4, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])   # scale 1: ties to even
    codes, scales = piq.int8_quantize_rows(x)
    c, s = S.quantize_rows_ref(f32(x))
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert scales[0] == 0 and scales[1] > 0 and scales[3] != scales[3]
    assert codes[4, :4].tolist() == [127, 0, 2, -2]


def linear_case(rng, tokens, inp, out, dtype, bias):
    x = rand(rng, (tokens, inp), dtype)
    w, ws = piq.int8_quantize_rows(rand(rng, (out, inp), FP32, 0.05))
    b = rand(rng, (out,), FP32) if bias else None
    return x, w, ws, b


def check_linear(y, x, w, ws, b):
    ref, prod = S.int8_linear_ref(f32(x), w.cpu().numpy(), f32(ws), None if b is None else f32(b))
    # three roundings of the product (from int32, two scales), one of the sum, all 2^-24,
    # and the rounding to the output's type
    tol = prod * 3.01 * 2.0 ** -24 + np.abs(ref) * (2.0 ** -24 + half_step(x.dtype) * 1.001) + 1e-30
    if x.dtype == FP16:
        tol += 2.0 ** -25    # half a step of its subnormal numbers
    assert worst(np.abs(f64(y) - ref), tol) <= 1


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("tokens,inp,out,bias", [
    (1, 8, 1, True), (1, 4096, 4096, True), (2, 1032, 130, False), (3, 24, 77, True),
    (4, 520, 999, False), (5, 264, 128, True), (8, 2056, 33, False), (9, 128, 257, True),
    (16, 1024, 512, True), (17, 136, 129, False), (31, 1032, 520, True), (64, 512, 384, False),
    (65, 776, 300, True), (127, 264, 128, True), (129, 2048, 260, False), (200, 72, 640, True),
    (256, 1024, 256, False), (300, 520, 1000, True), (515, 1288, 770, False)])
def test_int8_linear(tokens, inp, out, bias, dtype):
    rng = np.random.default_rng(tokens * inp + out)
    x, w, ws, b = linear_case(rng, tokens, inp, out, dtype, bias)
    check_linear(piq.int8_linear(x, w, ws, b), x, w, ws, b)


@pytest.mark.parametrize("tokens,inp,out", [(1, 28672, 520), (40, 28672, 300), (300, 11008, 640),
                                            (1030, 4104, 2050), (2100, 264, 2400)])
def test_int8_linear_long(tokens, inp, out):
    rng = np.random.default_rng(inp)
    x, w, ws, b = linear_case(rng, tokens, inp, out, BF16, True)
    check_linear(piq.int8_linear(x, w, ws, b), x, w, ws, b)


def test_int8_linear_largest_sums_are_exact():
    # every product 127 * 127 (and 127 * -128 of codes that no quantizer makes) over the
    # longest contraction: the int32 sum is exact up to its last bit
    inp = 131064
    for tokens in (1, 40, 300):
        x = torch.full((tokens, inp), 127.0, device="cuda")
        w = torch.full((48, (inp + 15) // 16 * 16), 127, dtype=torch.int8, device="cuda")[:, :inp]
        w[1] = -128
        w[2, 0] = 126
        y = piq.int8_linear(x, w, torch.ones(48, device="cuda"))
        ref = np.full((tokens, 48), 127.0 * 127 * inp)
        ref[:, 1] = -127.0 * 128 * inp
        ref[:, 2] -= 127
        assert np.array_equal(f32(y), ref.astype(np.float32))


@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_int8_linear_strides(tokens):
    # rows inside wider buffers, the result between columns that stay as they are
    rng = np.random.default_rng(tokens)
    x, w, ws, b = linear_case(rng, tokens, 520, 130, BF16, True)
    wide = torch.full((tokens, 600), float("nan"), dtype=BF16, device="cuda")
    wide[:, 40:560] = x
    ww = torch.full((130, 640), 99, dtype=torch.int8, device="cuda")
    ww[:, 16:536] = w
    y = torch.full((tokens + 1, 200), 7.0, dtype=BF16, device="cuda")
    got = piq.int8_linear(wide[:, 40:560], ww[:, 16:536], ws, b, out=y[:tokens, 3:133])
    assert got.data_ptr() == y[:, 3:].data_ptr()
    check_linear(y[:tokens, 3:133], x, w, ws, b)
    assert (y[tokens:] == 7).all() and (y[:, :3] == 7).all() and (y[:, 133:] == 7).all()


@pytest.mark.parametrize("tokens", [1, 6, 50, 200])
def test_int8_linear_bad_rows_stay_apart(tokens):
    rng = np.random.default_rng(tokens)
    x, w, ws, b = linear_case(rng, tokens, 264, 140, BF16, False)
    x[0, 7] = float("inf")
    y = piq.int8_linear(x, w, ws)
    assert torch.isnan(y[0]).all()
    if tokens > 1:
        check_linear(y[1:], x[1:], w, ws, None)
    x[0] = 0
    assert (piq.int8_linear(x, w, ws)[0] == 0).all()


def test_int8_linear_no_tokens():
    x, w, ws, b = linear_case(np.random.default_rng(0), 0, 64, 32, BF16, True)
    assert piq.int8_linear(x, w, ws, b).shape == (0, 32)


# --------------------------------------------------------------------------- cache
class Batch:
    """A ragged batch over a shuffled page table, in the library and in the oracle."""

    def __init__(self, rng, max_len, heads, dim, block, dtype, spare=2):
        self.rng, self.dtype, self.block = rng, dtype, block
        self.n = len(max_len)
        width = max(1, -(-max(max_len) // block)) + 1
        pages = self.n * width + spare
        self.table = rng.permutation(pages)[:self.n * width].reshape(self.n, width)
        self.cache = piq.kv8_cache(pages, heads, dim, block)
        self.ref = S.Kv8Ref(pages, heads, dim, block)
        self.lens = [0] * self.n
        self.shape = (heads, dim)
        # what lies in pages nobody wrote must not matter
        for i, t in enumerate(self.cache):
            t.fill_(float("nan") if i >= 2 else 77)
        for w in range(2):
            self.ref.codes[w][:] = 77
            self.ref.scale[w][:] = np.nan

    def gpu_table(self):
        wide = torch.full((self.n, self.table.shape[1] + 3), -5, dtype=torch.int32, device="cuda")
        wide[:, :self.table.shape[1]] = ints(self.table.tolist())
        return wide[:, :self.table.shape[1]]

    def append(self, news, std=1.0, fused=True, status=None):
        t, (h, d) = sum(news), self.shape
        cu = [0, *np.cumsum(news).tolist()]
        if fused:   # slices of one projection's output
            x = rand(self.rng, (t, 2 * h + 3, d), self.dtype, std)
            k, v = x[:, 1:1 + h], x[:, 2 + h:2 + 2 * h]
        else:
            k, v = (rand(self.rng, (t, h, d), self.dtype, std) for _ in range(2))
        piq.kv8_append(self.cache, k, v, ints(cu), ints(self.lens), self.gpu_table(),
                       status=status)
        self.ref.append((f32(k), f32(v)), cu, self.lens, self.table)
        self.lens = [a + b for a, b in zip(self.lens, news)]

    def check(self):
        for w in range(2):
            assert np.array_equal(self.cache[w].cpu().numpy(), self.ref.codes[w])
            assert np.array_equal(self.cache[2 + w].cpu().numpy(), self.ref.scale[w],
                                  equal_nan=True)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_append_is_the_definition(dtype, dim, block):
    # whole caches compared: codes, scales, and what no call may touch
    rng = np.random.default_rng(block + dim)
    b = Batch(rng, [400, 300, 0, 300, 33], 3, dim, block, dtype)
    for news, std in (([1, 0, 0, 17, 0], 1.0), ([1, 1, 0, 1, 0], 3.0), ([block, 200, 0, 3, 33], 2.0),
                      ([129, 1, 0, 64, 0], 0.1), ([1, 1, 0, 1, 0], 9.0)):
        b.append(news, std)
        b.check()


def test_append_many_sequences_and_no_tokens():
    rng = np.random.default_rng(3)
    b = Batch(rng, [40] * 200, 1, 64, 16, BF16)
    for news in ([1] * 200, [0] * 200, rng.integers(0, 12, 200).tolist(), [1] * 200):
        b.append(news, fused=False)
        b.check()


def test_append_zero_and_bad_values():
    rng = np.random.default_rng(4)
    b = Batch(rng, [64], 2, 64, 32, FP32)
    b.append([5], std=0.0)       # a block of zeros: scale 0
    b.check()
    b.append([3], std=1.0)       # then values: the zeros stay zeros
    b.check()
    k = torch.ones(1, 2, 64, device="cuda")
    k[0, 1, 3] = float("inf")
    piq.kv8_append(b.cache, k, k, ints([0, 1]), ints([8]), b.gpu_table())
    b.ref.append((f32(k), f32(k)), [0, 1], [8], b.table)
    b.lens = [9]
    b.check()                    # head 1's block has scale NaN, head 0 does not
    assert torch.isnan(b.cache.k_scale[b.table[0][0]]).tolist() == [False, True]
    b.append([2])
    b.check()                    # and keeps it until its first token is written again
    b.lens = [0]
    b.append([4])
    b.check()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64)])
def test_read_back(dtype, dim, block):
    rng = np.random.default_rng(5)
    b = Batch(rng, [100, 70, 5, 90], 3, dim, block, FP32)
    b.append([100, 70, 5, 90])
    start, stop = [3, 70, 0, 17], [100, 70, 5, 18]
    cu = [2, *(2 + np.cumsum([e - s for s, e in zip(start, stop)])).tolist()]
    rows = cu[-1] + 2            # rows before the first and behind the last sequence
    outs = tuple(torch.full((rows, 4, dim), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    piq.kv8_read(b.cache, ints(cu), ints(start), b.gpu_table(), rows, dtype,
                 out=tuple(o[:, :3] for o in outs))
    for w, o in enumerate(outs):
        got = f64(o)
        assert (got[:2] == 5).all() and (got[cu[-1]:] == 5).all() and (got[:, 3] == 5).all()
        for i in range(4):
            ref = b.ref.tokens(w, i, start[i], stop[i], b.table)
            tol = np.abs(ref) * (2.0 ** -24 + half_step(dtype) * 1.001) + 2.0 ** -25
            assert worst(np.abs(got[cu[i]:cu[i + 1], :3] - ref), tol) <= 1


def test_bad_pages_and_lengths_are_reported():
    rng = np.random.default_rng(6)
    b = Batch(rng, [40, 40, 40], 2, 64, 16, BF16)
    status = piq.new_status()
    b.append([20, 20, 20], status=status)
    assert status.tolist() == [0, 0]
    table = b.gpu_table().clone()
    table[1, 1] = 10 ** 6
    cu, lens = ints([0, 1, 2, 3]), ints([20, 20, 20])
    before = [t.clone() for t in b.cache]
    kv = rand(rng, (3, 2, 64), BF16)
    piq.kv8_append(b.cache, kv, kv, cu, lens, table, status=status)
    assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 1]
    with pytest.raises(piq.PiqError):
        piq.check_status(status)
    assert status.tolist() == [0, 0]
    b.ref.append((f32(kv)[[0, 2]],) * 2, [0, 1, 2], [20, 20], b.table[[0, 2]])
    b.check()                                    # the other two were written, nothing else
    # reading and attending: the bad sequence is NaN, the others are what they were
    k, v = piq.kv8_read(b.cache, ints([0, 20, 40, 60]), ints([0, 0, 0]), table, 60, status=status)
    assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 1]
    assert torch.isnan(k[36:40]).all() and not torch.isnan(k[:36]).any() and \
        not torch.isnan(k[40:]).any()
    status.zero_()
    q = rand(rng, (3, 4, 64), BF16)
    good = piq.kv8_attention(b.cache, q, cu, ints([21, 20, 21]), b.gpu_table(), 1, 21)
    out = piq.kv8_attention(b.cache, q, cu, ints([21, 20, 21]), table, 1, 21, status=status)
    assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 1]
    assert torch.isnan(out[1]).all() and torch.equal(out[[0, 2]], good[[0, 2]])
    # lengths out of range: longer than the table, than max_len, fewer than the new tokens
    for bad in (10 ** 6, 22, 0, -4):
        status.zero_()
        out, lse = piq.kv8_attention(b.cache, q, cu, ints([21, bad, 21]), b.gpu_table(), 1, 21,
                                     return_lse=True, status=status)
        assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 1]
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
        assert torch.equal(out[[0, 2]], good[[0, 2]])
    status.zero_()
    before = [t.clone() for t in b.cache]
    for bad in (-1, 10 ** 6):
        piq.kv8_append(b.cache, kv[:1], kv[:1], ints([0, 0, 1, 1]), ints([21, bad, 21]),
                       b.gpu_table(), status=status)
        assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 1]
    piq.kv8_append(b.cache, kv[:1], kv[:1], ints([0, 0, 5, 5]), ints([21, 20, 21]),
                   b.gpu_table(), status=status)   # more rows than there are
    for x, y in zip(before, b.cache):
        assert torch.equal(x.view(torch.int8), y.view(torch.int8))


# ----------------------------------------------------------------------- attention
def check_attention(b, q, news, out, lse, window=0, scale=None):
    cu = [0, *np.cumsum(news).tolist()]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    ref, rl, tol, tol_l = S.attention_ref(b.ref, f64(q), cu, b.lens, b.table, scale, window)
    got, gl = f64(out), f64(lse)
    tol = tol + np.abs(ref) * half_step(q.dtype) * 1.01 + 2.0 ** -25
    fine = np.isfinite(f64(q)).all(2)          # a query row with an infinity is NaN
    assert np.isnan(got[~fine]).all() and np.isnan(gl[~fine]).all()
    assert worst(np.abs(got - ref)[fine], tol[fine]) <= 1
    seen = fine & np.isfinite(rl)
    assert (gl[fine & ~seen] == -np.inf).all()
    assert worst(np.abs(gl - rl)[seen], tol_l[seen]) <= 1


def run_attention(b, q, news, max_len=None, window=0, **kw):
    cu = [0, *np.cumsum(news).tolist()]
    return piq.kv8_attention(b.cache, q, ints(cu), ints(b.lens), b.gpu_table(),
                             max(news), max_len or max(b.lens), window=window, return_lse=True,
                             **kw)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 2), (6, 2), (16, 1), (40, 2)])
def test_attention_one_token(dtype, dim, block, heads, kv_heads):
    rng = np.random.default_rng(heads + dim + block)
    b = Batch(rng, [1, 700, 129, 16, 17, 3, 300], kv_heads, dim, block, dtype)
    b.append([0, 690, 128, 15, 16, 0, 299])
    news = [1, 1, 1, 1, 1, 0, 1]
    b.append(news)
    q = rand(rng, (sum(news), heads, dim), dtype, 2.0)
    check_attention(b, q, news, *run_attention(b, q, news))


@pytest.mark.parametrize("news,lens", [([3], [3]), ([2, 5, 1], [40, 5, 300]),
                                       ([70, 1, 130], [200, 129, 130]), ([257], [400])])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 64), (8, 2, 128), (12, 1, 128)])
@pytest.mark.parametrize("window", [0, 1, 37, 128])
def test_attention_chunks_of_new_tokens(news, lens, heads, kv_heads, dim, window):
    rng = np.random.default_rng(sum(lens) + heads)
    b = Batch(rng, lens, kv_heads, dim, 32, FP16)
    b.append([a - n for a, n in zip(lens, news)])
    b.append(news)
    q = rand(rng, (sum(news), heads, dim), FP16, 1.5)
    check_attention(b, q, news, *run_attention(b, q, news, window=window), window=window)


@pytest.mark.parametrize("max_len", [5000, 100000])
@pytest.mark.parametrize("news,window", [([1, 1, 1], 0), ([1, 0, 1], 900), ([2, 40, 3], 0)])
def test_attention_split_and_joined(max_len, news, window):
    # a bound far above the lengths, and lengths of one chunk and of many in one batch
    rng = np.random.default_rng(7)
    b = Batch(rng, [4990, 60, 1500], 2, 64, 64, BF16)
    b.append([4000, 20, 1400])
    b.append(news)
    q = rand(rng, (sum(news), 6, 64), BF16, 2.0)
    check_attention(b, q, news, *run_attention(b, q, news, max_len, window), window=window)


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,block,news,lens,window", [
    (BF16, 4, 1, 128, 16, [300], [1500], 0), (BF16, 8, 4, 64, 128, [260, 90], [700, 1300], 0),
    (FP16, 2, 2, 128, 64, [513], [513], 0), (BF16, 16, 2, 128, 32, [40, 3, 200], [900, 2000, 210], 333),
    (FP16, 64, 2, 64, 64, [20, 9], [1100, 70], 0)])
def test_attention_prompts(dtype, heads, kv_heads, dim, block, news, lens, window):
    # several tiles of rows and of keys, scales that move between blocks
    rng = np.random.default_rng(heads * block)
    b = Batch(rng, lens, kv_heads, dim, block, dtype)
    half = [(a - n) // 2 for a, n in zip(lens, news)]
    b.append(half, std=0.2)
    b.append([a - n - h for a, n, h in zip(lens, news, half)], std=3.0)
    b.append(news)
    q = rand(rng, (sum(news), heads, dim), dtype, 1.5)
    check_attention(b, q, news, *run_attention(b, q, news, window=window), window=window)
    big = max(lens) * 40          # a bound that splits the keys of few rows
    check_attention(b, q, news, *run_attention(b, q, news, big, window), window=window)


def test_attention_negative_scale():
    rng = np.random.default_rng(17)
    b = Batch(rng, [200, 90], 2, 64, 32, BF16)
    b.append([190, 30])
    for news in ([1, 1], [9, 59]):
        b.append(news)
        q = rand(rng, (sum(news), 8, 64), BF16)
        check_attention(b, q, news, *run_attention(b, q, news, scale=-0.3), scale=-0.3)


def test_attention_rows_and_strides():
    rng = np.random.default_rng(8)
    b = Batch(rng, [70, 9], 2, 64, 16, BF16)
    b.append([60, 4])
    news = [3, 1]
    b.append(news)
    wide = torch.full((6, 9, 64), float("nan"), dtype=BF16, device="cuda")
    q = rand(rng, (4, 4, 64), BF16)
    wide[:4, 2:6] = q
    out = torch.full((6, 5, 64), 3.0, dtype=BF16, device="cuda")
    cu = ints([0, 3, 4])
    piq.kv8_attention(b.cache, wide[:, 2:6], cu, ints(b.lens), b.gpu_table(), 3, 70,
                      out=out[:, 1:])
    _, lse = run_attention(b, q, news)
    check_attention(b, q, news, out[:4, 1:], lse)
    assert (out[4:] == 3).all() and (out[:, 0] == 3).all()   # rows of no sequence, other columns


def test_attention_large_scores_and_scales():
    # scores of thousands, value scales that differ by 2^20 between blocks
    rng = np.random.default_rng(9)
    b = Batch(rng, [200], 1, 64, 16, FP32)
    for i in range(12):
        b.append([16], std=2.0 ** (10 - 20 * (i % 2)))
    news = [1]
    b.append(news)
    for std in (1e-6, 1.0, 100.0):
        q = rand(rng, (1, 4, 64), BF16, std)
        check_attention(b, q, news, *run_attention(b, q, news))


@pytest.mark.parametrize("dtype,big,small", [(BF16, 2.0 ** 100, 2.0 ** -120), (FP16, 6e4, 6e-8)])
def test_attention_extreme_queries(dtype, big, small):
    rng = np.random.default_rng(10)
    b = Batch(rng, [50], 1, 64, 16, FP32)
    b.append([49], std=1e-3)
    b.append([1], std=1e-3)
    q = rand(rng, (1, 3, 64), dtype)
    q[0, 0] *= small
    q[0, 1] *= big
    q[0, 2] = 0
    scale = 0.1 / big
    check_attention(b, q, [1], *run_attention(b, q, [1], scale=scale), scale=scale)
    q[0, 1, 5] = float("inf")
    out, lse = run_attention(b, q, [1], scale=scale)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert not torch.isnan(out[0, [0, 2]]).any()


def test_attention_bad_block_out_of_sight():
    # a NaN block outside a window, or behind a query, does not reach it
    rng = np.random.default_rng(11)
    b = Batch(rng, [300], 1, 64, 16, BF16)
    b.append([290])
    page = int(b.table[0][2])
    b.cache.k_scale[page] = b.cache.v_scale[page] = float("nan")
    b.ref.scale[0][page] = b.ref.scale[1][page] = np.nan
    news = [4]
    b.append(news)
    q = rand(rng, (4, 2, 64), BF16)
    out, lse = run_attention(b, q, news, window=200)
    check_attention(b, q, news, out, lse, window=200)
    assert torch.isnan(run_attention(b, q, news)[0]).all()


# ------------------------------------------------------------- streams, graphs, one layer
def layer(b, x, wqkv, wo, cu, lens, table, heads, max_new, max_len):
    """One attention layer in 8 bits: projection, cache, attention, projection."""
    kvh, dim = b.shape
    qkv = piq.int8_linear(x, *wqkv).view(-1, heads + 2 * kvh, dim)
    piq.kv8_append(b.cache, qkv[:, heads:heads + kvh], qkv[:, heads + kvh:], cu, lens, table)
    now = lens + (cu[1:] - cu[:-1])
    o = piq.kv8_attention(b.cache, qkv[:, :heads], cu, now, table, max_new, max_len)
    return qkv, o, piq.int8_linear(o.view(-1, heads * dim), *wo)


def layer_case(seed):
    rng = np.random.default_rng(seed)
    heads, kvh, dim, model = 8, 2, 64, 264
    b = Batch(rng, [90, 40, 200], kvh, dim, 32, BF16)
    wqkv = piq.int8_quantize_rows(rand(rng, ((heads + 2 * kvh) * dim, model), FP32, 0.08))
    wo = piq.int8_quantize_rows(rand(rng, (model, heads * dim), FP32, 0.08))
    return rng, b, wqkv, wo, heads, model


def check_layer(b, x, qkv, o, y, wqkv, wo, news, heads):
    kvh, dim = b.shape
    check_linear(qkv.reshape(len(x), -1), x, *wqkv, None)
    cu = [0, *np.cumsum(news).tolist()]
    b.ref.append((f32(qkv[:, heads:heads + kvh]), f32(qkv[:, heads + kvh:])), cu, b.lens, b.table)
    b.lens = [a + n for a, n in zip(b.lens, news)]
    b.check()
    ref, _, tol, _ = S.attention_ref(b.ref, f64(qkv[:, :heads]), cu, b.lens, b.table, dim ** -0.5)
    tol = tol + np.abs(ref) * half_step(BF16) * 1.01
    assert worst(np.abs(f64(o) - ref), tol) <= 1
    check_linear(y, o.reshape(len(x), -1), *wo, None)


def test_one_layer_prompt_then_steps():
    rng, b, wqkv, wo, heads, model = layer_case(12)
    for news in ([50, 1, 130], [1, 1, 1], [1, 0, 1], [3, 30, 1]):
        x = rand(rng, (sum(news), model), BF16)
        cu = ints([0, *np.cumsum(news).tolist()])
        out = layer(b, x, wqkv, wo, cu, ints(b.lens), b.gpu_table(), heads, max(news), 200)
        check_layer(b, x, *out, wqkv, wo, news, heads)


def test_one_layer_captured_step():
    # a decoding step captured once and replayed with new inputs, lengths and cache contents
    rng, b, wqkv, wo, heads, model = layer_case(13)
    b.append([70, 20, 150])
    x = torch.zeros(3, model, dtype=BF16, device="cuda")
    cu, lens, table = ints([0, 1, 2, 3]), ints(b.lens), b.gpu_table()
    saved = [t.clone() for t in b.cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(b, x, wqkv, wo, cu, lens, table, heads, 1, 200)   # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(b, x, wqkv, wo, cu, lens, table, heads, 1, 200)
        lens += 1
    for t, s in zip(b.cache, saved):
        t.copy_(s)
    for _ in range(4):
        x.copy_(rand(rng, (3, model), BF16))
        graph.replay()
        torch.cuda.synchronize()
        check_layer(b, x, *out, wqkv, wo, [1, 1, 1], heads)
        assert lens.tolist() == b.lens


def test_streams_side_by_side():
    # two streams at once with workspaces of their own give what one after the other gives
    rng = np.random.default_rng(14)
    b = Batch(rng, [3000, 2000], 2, 64, 64, BF16)
    b.append([2999, 1999])
    b.append([1, 1])
    q = rand(rng, (2, 8, 64), BF16)
    x, w, ws, bias = linear_case(rng, 40, 2056, 520, BF16, True)
    want = run_attention(b, q, [1, 1], 100000)[0], piq.int8_linear(x, w, ws, bias)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        for s in streams:
            got.append((run_attention(b, q, [1, 1], 100000, stream=s)[0],
                        piq.int8_linear(x, w, ws, bias, stream=s)))
    torch.cuda.synchronize()
    for a, c in got:
        assert torch.equal(a, want[0]) and torch.equal(c, want[1])


def test_results_repeat_bit_for_bit():
    rng = np.random.default_rng(15)
    b = Batch(rng, [900, 2500], 2, 128, 64, FP16)
    b.append([700, 2400])
    news = [150, 60]
    b.append(news)
    q = rand(rng, (210, 8, 128), FP16)
    first = run_attention(b, q, news)
    for _ in range(5):
        again = run_attention(b, q, news)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refuses_what_does_not_fit():
    rng = np.random.default_rng(16)
    x, w, ws, b = linear_case(rng, 4, 64, 32, BF16, True)
    with pytest.raises(ValueError):
        piq.int8_linear(x[:, :56], w, ws)
    with pytest.raises(ValueError):
        piq.int8_linear(x, w, ws[:31])
    with pytest.raises(TypeError):
        piq.int8_linear(x.double(), w, ws)
    with pytest.raises(ValueError):
        piq.int8_linear(x.t(), w, ws)
    with pytest.raises(ValueError):
        piq.int8_linear(x, w, ws, out=torch.empty(4, 33, dtype=BF16, device="cuda"))
    c = piq.kv8_cache(4, 2, 64, 16)
    cu, lens, table = ints([0, 1]), ints([0]), ints([[0, 1]])
    kv = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        piq.kv8_append(c, kv[:, :1], kv[:, :1], cu, lens, table)
    with pytest.raises(ValueError):
        piq.kv8_append(c, kv, kv, ints([0, 0, 1]), lens, table)
    with pytest.raises(TypeError):
        piq.kv8_append(c, kv, kv, cu, lens, table.long())
    with pytest.raises(TypeError):
        piq.kv8_attention(c, kv.float(), cu, lens, table, 1, 1)
    with pytest.raises(ValueError):
        piq.kv8_attention(c, torch.zeros(1, 2, 128, dtype=BF16, device="cuda"), cu, lens, table,
                          1, 1)
    with pytest.raises(piq.PiqError):
        piq.kv8_attention(c, torch.zeros(1, 3, 64, dtype=BF16, device="cuda"), cu, lens, table,
                          1, 1)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,new", [(17, 1), (8, 3), (8, 4), (11, 3), (8, 5), (16, 3), (7, 7),
                                       (32, 2)])
def test_attention_where_the_kernels_meet(dtype, dim, group, new):
    # rows a kv head from 17 to 64: groups of rows on one side, one tile of them on the other
    rng = np.random.default_rng(100 * group + new)
    b = Batch(rng, [700, 90, 330], 2, dim, 32, dtype)
    b.append([650, 10, 300])
    news = [new, 1, max(new - 1, 1)]
    b.append(news)
    q = rand(rng, (sum(news), 2 * group, dim), dtype)
    for window, max_len in ((0, max(b.lens)), (100, max(b.lens)), (0, 40000)):
        out, lse = run_attention(b, q, news, max_len, window)
        check_attention(b, q, news, out, lse, window)


@pytest.mark.parametrize("heads,news", [(4, [1, 2, 1]), (8, [30, 64, 20])])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_bad_page_reaches_its_readers_only(dim, heads, news):
    # a bad page in the middle of one sequence's new tokens: queries before it see nothing of it
    rng = np.random.default_rng(21)
    b = Batch(rng, [200, 200, 200], 2, dim, 16, BF16)
    b.append([100, 127, 90])
    b.append(news)
    q = rand(rng, (sum(news), heads, dim), BF16)
    good, _ = run_attention(b, q, news)
    table = b.gpu_table().clone()
    table[1, 128 // 16] = -7                       # positions 128 ..; the new ones start at 127
    status = piq.new_status()
    cu = [0, *np.cumsum(news).tolist()]
    out = piq.kv8_attention(b.cache, q, ints(cu), ints(b.lens), table, max(news), max(b.lens),
                            status=status)
    assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 1]
    first = cu[1] + 1
    assert torch.isnan(out[first:cu[2]]).all()
    keep = [i for i in range(sum(news)) if not first <= i < cu[2]]
    assert torch.isfinite(out[keep]).all()
    # the value scales of the page are gone too, so the scaling of probabilities may move:
    # their roundings, 2^-11 on either side, of values below 8, and one of the result each
    assert worst(np.abs(f64(out[keep]) - f64(good[keep])),
                 np.abs(f64(good[keep])) * 2.02 * half_step(BF16) + 2.0 ** -7) <= 1


def test_rows_of_no_sequence_and_no_new_tokens():
    rng = np.random.default_rng(22)
    b = Batch(rng, [40, 40], 2, 64, 16, BF16)
    b.append([20, 30])
    q = rand(rng, (5, 4, 64), BF16)
    out = torch.full_like(q, 7.0)
    status = piq.new_status()
    piq.kv8_attention(b.cache, q, ints([0, 0, 0]), ints(b.lens), b.gpu_table(), 0, 40, out=out,
                      status=status)
    assert (out == 7).all() and status.tolist() == [0, 0]
    # max_new below what the lengths say is an error, not silence
    piq.kv8_attention(b.cache, q, ints([0, 1, 1]), ints(b.lens), b.gpu_table(), 0, 40, out=out,
                      status=status)
    assert torch.isnan(out[0]).all() and (out[1:] == 7).all()
    assert status.tolist() == [piq.PIQ_ERR_INVALID_ARG, 0]
    with pytest.raises(piq.PiqError):
        piq.kv8_attention(b.cache, q, ints([0, 1, 1]), ints(b.lens), b.gpu_table(), 1, 40,
                          scale=3e38)


def test_captured_calls_of_every_kernel():
    # prompts back to back, split and joined keys and every form of the product, captured
    # twice with workspaces of their own and replayed side by side on new inputs
    rng = np.random.default_rng(23)
    b = Batch(rng, [1200, 3000], 2, 128, 64, BF16)
    b.append([900, 2800])
    b.append([100, 90])
    q = torch.zeros(190, 8, 128, dtype=BF16, device="cuda")
    step = torch.zeros(2, 8, 128, dtype=BF16, device="cuda")
    lin = [linear_case(rng, t, 1032, 520, BF16, True) for t in (1, 30, 200, 1500)]
    cu, one, lens, table = ints([0, 100, 190]), ints([0, 1, 2]), ints(b.lens), b.gpu_table()

    def work():
        got = [piq.kv8_attention(b.cache, q, cu, lens, table, 100, 3000) for _ in range(2)]
        got.append(piq.kv8_attention(b.cache, step, one, lens, table, 1, 100000))
        return got + [piq.int8_linear(*c) for c in lin]

    work()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work())
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        q.copy_(rand(rng, q.shape, BF16))
        step.copy_(rand(rng, step.shape, BF16))
        for c in lin:
            c[0].copy_(rand(rng, c[0].shape, BF16))
        want = work()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for got in outs:
            for x, y in zip(got, want):
                assert torch.equal(x, y)


def test_default_stream_given_by_handle():
    rng = np.random.default_rng(24)
    x, w, ws, bias = linear_case(rng, 9, 520, 264, FP16, True)
    want = piq.int8_linear(x, w, ws, bias)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                  # another stream is current
        got = piq.int8_linear(x, w, ws, bias, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_quantized_weights_used_at_once():
    # the product asks for the weights before the kernels ahead of it end, but not before
    # the one that writes them has ended
    rng = np.random.default_rng(25)
    x = rand(rng, (40, 4096), BF16)
    for i in range(10):
        w = rand(rng, (1024, 4096), BF16)
        torch.cuda.synchronize()
        codes, scale = piq.int8_quantize_rows(w)
        y = piq.int8_linear(x, codes, scale)
        torch.cuda.synchronize()
        assert torch.equal(y, piq.int8_linear(x, codes, scale))


@pytest.mark.parametrize("heads,kv_heads,dim,block,news,lens,window", [
    (1, 1, 64, 128, [226, 132], [1224, 221], 240), (2, 2, 128, 128, [226, 100], [1224, 1000], 240),
    (4, 1, 64, 32, [100, 64, 30], [1500, 900, 1111], 333), (8, 2, 128, 16, [70], [2000], 777),
    (8, 1, 64, 64, [9, 200], [3000, 2500], 1500)])
def test_attention_window_over_split_keys(heads, kv_heads, dim, block, news, lens, window):
    # the window's first key is not on the grid of the parts that the keys are split into
    rng = np.random.default_rng(sum(lens) + window)
    b = Batch(rng, [n + 50 for n in lens], kv_heads, dim, block, BF16)
    b.append([total - n for total, n in zip(lens, news)])
    b.append(news)
    q = rand(rng, (sum(news), heads, dim), BF16)
    for w in (window, window + 1, window + 64):
        out, lse = run_attention(b, q, news, window=w)
        check_attention(b, q, news, out, lse, w)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_new", [1, 100])
def test_attention_score_beside_loud_query_channels(dtype, dim, max_new):
    # One key a query, so lse is its score, a small integer: queries that are loud where the
    # key is 0 must not take bits from it.  Codes and queries are integers (the largest key is
    # 127: its scale is 1) and the sum is exact in fp32, so the score is off by the roundings
    # of scale log2(e) (2), of the two products with it and of ln 2 and the product with that:
    # at most 6 of 2^-24, and second-order terms.  (max_new picks the kernel.)
    rng = np.random.default_rng(31)
    n = 60
    k, q = np.zeros((n, 1, dim), np.float32), np.zeros((n, 2, dim), np.float32)
    k[:, 0, :8] = rng.integers(-9, 10, (n, 8))
    k[:, 0, 0] = 127
    q[..., :8] = rng.integers(1, 4, (n, 2, 8))
    q[..., 8:] = 1024 + 8 * rng.integers(0, 64, (n, 2, dim - 8))
    cache = piq.kv8_cache(n, 1, dim, 16)
    kt, qt = (torch.from_numpy(a).cuda().to(dtype) for a in (k, q))
    cu, table = ints(list(range(n + 1))), ints([[i] for i in range(n)])
    piq.kv8_append(cache, kt, kt, cu, ints([0] * n), table)
    assert (cache.k_scale == 1).all()
    out, lse = piq.kv8_attention(cache, qt, cu, ints([1] * n), table, max_new, 1,
                                 return_lse=True)
    want = (q.astype(np.float64) * k).sum(2) * dim ** -0.5
    assert (np.abs(f64(lse) - want) <= 6.1 * 2.0 ** -24 * np.abs(want)).all()
    assert torch.equal(out, kt.expand(n, 2, dim))


# ---------------------------------------------------------- values far apart in size
def put(b, news, k, v):
    """Appends the given keys and values (fp32 [tokens, heads, dim]) on both sides."""
    cu = [0, *np.cumsum(news).tolist()]
    k, v = np.ascontiguousarray(k, np.float32), np.ascontiguousarray(v, np.float32)
    piq.kv8_append(b.cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), ints(cu),
                   ints(b.lens), b.gpu_table())
    b.ref.append((k, v), cu, b.lens, b.table)
    b.lens = [x + n for x, n in zip(b.lens, news)]


def check_sizes(b, q, news, out, lse, window=0):
    """check_attention for bf16 results of any size: the smallest steps are bf16's, 2^-133."""
    cu = [0, *np.cumsum(news).tolist()]
    ref, rl, tol, tol_l = S.attention_ref(b.ref, f64(q), cu, b.lens, b.table, q.shape[2] ** -0.5,
                                          window)
    assert out.dtype == BF16
    tol = tol + np.abs(ref) * half_step(BF16) * 1.01 + 2.0 ** -134
    assert worst(np.abs(f64(out) - ref), tol) <= 1
    assert worst(np.abs(f64(lse) - rl), tol_l) <= 1


BOTH = [(4, 1), (4, 4), (8, 60)]    # heads and new tokens: groups of rows, tiles of rows


@pytest.mark.parametrize("heads,new", BOTH)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tiny", [400, 320, 32, 1])
def test_attention_smallest_value_scales(dim, heads, new, tiny):
    # value scales from the smallest that are kept, 2^-126, in the first blocks or in all
    rng = np.random.default_rng(dim + tiny)
    b = Batch(rng, [400], 1, dim, 16, FP32)
    k, v = rng.normal(0, 1, (2, 400, 1, dim)).astype(np.float32)
    small = slice(0, -(-tiny // 16) * 16)
    v[small] *= 3e-37
    v[small][::16, 0, 5] = 1.6e-36          # each block's largest: above 127 * 2^-126
    put(b, [400 - new], k[:400 - new], v[:400 - new])
    put(b, [new], k[400 - new:], v[400 - new:])
    first = b.ref.scale[1][b.table[0][0]]
    assert 2.0 ** -126 <= first[0] < 2.0 ** -124
    q = rand(rng, (new, heads, dim), BF16)
    for max_len in (400, 40000):
        check_sizes(b, q, [new], *run_attention(b, q, [new], max_len))


@pytest.mark.parametrize("heads,new", [(4, 4), (8, 60)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 208])
@pytest.mark.parametrize("big", [2.0 ** 14, 2.0 ** 40, 2.0 ** 100])
def test_attention_values_out_of_sight(dim, heads, new, window, big):
    # Blocks of large values that only some rows see, behind the others' position (no window)
    # or before their window: the others are as exact as without them, and the same to the bit.
    rng = np.random.default_rng(dim + window)
    b = Batch(rng, [386], 1, dim, 16, FP32)
    k, v = rng.normal(0, 1, (2, 386, 1, dim)).astype(np.float32)
    large = slice(0, 176) if window else slice(384, 386)
    v[large] *= big
    put(b, [386 - new], k[:386 - new], v[:386 - new])
    put(b, [new], k[386 - new:], v[386 - new:])
    q = rand(rng, (new, heads, dim), BF16)
    pos = np.arange(386 - new, 386)
    blind = (pos - window + 1 >= 176) if window else pos < 384
    assert 0 < blind.sum() < new
    for max_len in (386, 40000):
        out, lse = run_attention(b, q, [new], max_len, window)
        check_sizes(b, q, [new], out, lse, window)


@pytest.mark.parametrize("heads,new", BOTH)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1e33, 1e37, 3e38])
def test_attention_largest_values(dim, heads, new, size):
    # averages of values near fp32's largest: no sum on the way is larger than they are
    rng = np.random.default_rng(dim)
    b = Batch(rng, [1000], 1, dim, 32, FP32)
    k = rng.normal(0, 0.1, (1000, 1, dim)).astype(np.float32)
    v = (size * rng.uniform(0.9, 1.0, (1000, 1, dim))).astype(np.float32)
    put(b, [1000 - new], k[:1000 - new], v[:1000 - new])
    put(b, [new], k[1000 - new:], v[1000 - new:])
    q = rand(rng, (new, heads, dim), BF16)
    for max_len in (1000, 100000):
        check_sizes(b, q, [new], *run_attention(b, q, [new], max_len))


# ---------------------------------------------------------------- waits that give up
def linear_call(tokens, inp, out):
    rng = np.random.default_rng(tokens)
    x, w, ws, bias = linear_case(rng, tokens, inp, out, BF16, True)
    y = torch.empty(tokens, out, dtype=BF16, device="cuda")
    return lambda status: (piq.int8_linear(x, w, ws, bias, out=y, status=status),)


def attention_call(heads, kv_heads, dim, batch, new, length, max_len):
    g = torch.Generator(device="cuda").manual_seed(heads)
    pages = -(-length // 64)
    shape = (batch * pages, kv_heads, 64, dim)
    codes = [torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
             for _ in range(2)]
    scales = [torch.rand(shape[:2], generator=g, device="cuda") / 50 for _ in range(2)]
    cache = piq.KV8Cache(*codes, *scales)
    table = torch.randperm(shape[0], generator=g, device="cuda").int().view(batch, pages)
    q = torch.randn(batch * new, heads, dim, generator=g, device="cuda").to(BF16)
    cu, lens = ints([new * i for i in range(batch + 1)]), ints([length] * batch)
    return lambda status: piq.kv8_attention(cache, q, cu, lens, table, new, max_len,
                                            return_lse=True, status=status)


@pytest.mark.parametrize("call,args", [
    (linear_call, (300, 1032, 2050)),            # one slice of k
    (linear_call, (37, 11008, 4096)),            # eight, joined in a cluster
    (linear_call, (2100, 4104, 4000)),           # pairs of CTAs, several tiles each
    (attention_call, (32, 8, 128, 32, 1, 4096, 4096)),      # groups of rows
    (attention_call, (16, 8, 64, 4, 1, 50000, 50000)),    # split and joined
    (attention_call, (32, 2, 128, 4, 300, 2000, 2000)),     # tiles of rows
    (attention_call, (8, 1, 64, 2, 60, 3000, 60000))])      # split and joined
def test_a_wait_that_gives_up_leaves_nan(call, args):
    # the shortest limit: what a wait was given up for is NaN, the rest as it should be, the
    # status says so, and the next call is what it was
    run = call(*args)
    want, status = [t.clone() for t in run(None)], piq.new_status()
    seen = 0
    try:
        for _ in range(5):
            status.zero_()
            piq.serving_wait_limit(1)
            got = run(status)
            torch.cuda.synchronize()
            piq.serving_wait_limit(0)
            code = status.tolist()[0]
            assert code in (piq.PIQ_OK, piq.PIQ_ERR_TIMEOUT)
            seen += code != piq.PIQ_OK
            for g, w in zip(got, want):
                nan = torch.isnan(g)
                assert torch.equal(g[~nan], w[~nan])
                assert code == piq.PIQ_ERR_TIMEOUT or not nan.any()
    finally:
        piq.serving_wait_limit(0)
    assert seen
    status.zero_()
    for g, w in zip(run(status), want):
        assert torch.equal(g, w)
    assert status.tolist() == [0, 0]


# ------------------------------------------------------------------- bad row starts
BAD_STARTS = [[-5000, 10], [-1, 4, 10], [10 ** 6, 10 ** 6 + 1], [0, 5, 3], [0, 4, 12],
              [11, 12, 13], [0, 10, 2 ** 31 - 1, -2 ** 31], [-2 ** 31, -2 ** 31]]


def bad_sequences(cu, rows):
    return [i for i in range(len(cu) - 1)
            if not 0 <= cu[i] <= cu[i + 1] <= rows and cu[i] != cu[i + 1]]


@pytest.mark.parametrize("cu", BAD_STARTS)
@pytest.mark.parametrize("heads", [2, 16, 200])
def test_attention_bad_starts_are_reported(cu, heads):
    # whatever the kernel (heads of 2 kv heads pick it) and wherever the rows would lie
    rng = np.random.default_rng(heads)
    n, bad = len(cu) - 1, bad_sequences(cu, 10)
    b = Batch(rng, [60] * n, 2, 64, 16, BF16)
    b.append([60] * n)
    q = rand(rng, (10, heads, 64), BF16)
    status, out = piq.new_status(), torch.full_like(q, 3.0)
    _, lse = piq.kv8_attention(b.cache, q, ints(cu), ints(b.lens), b.gpu_table(), 10, 60,
                               out=out, return_lse=True, status=status)
    assert bool(bad) == (status.tolist()[0] == piq.PIQ_ERR_INVALID_ARG)
    if bad:
        assert status.tolist()[1] in bad
    for i in bad:
        rows = slice(max(cu[i], 0), max(min(cu[i + 1], 10), 0))
        assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()


@pytest.mark.parametrize("cu", BAD_STARTS)
def test_append_and_read_bad_starts_are_reported(cu):
    rng = np.random.default_rng(1)
    n, bad = len(cu) - 1, bad_sequences(cu, 10)
    b = Batch(rng, [80] * n, 2, 64, 16, BF16)
    b.append([40] * n)
    kv = rand(rng, (10, 2, 64), BF16)
    status, before = piq.new_status(), [t.clone() for t in b.cache]
    piq.kv8_append(b.cache, kv, kv, ints(cu), ints(b.lens), b.gpu_table(), status=status)
    assert bool(bad) == (status.tolist()[0] == piq.PIQ_ERR_INVALID_ARG)
    for i in bad:                                  # their pages are as they were
        assert status.tolist()[1] in bad
        for x, y in zip(before, b.cache):
            p = torch.from_numpy(b.table[i].copy()).cuda()
            assert torch.equal(x[p].view(torch.int8), y[p].view(torch.int8))
    status.zero_()
    out = tuple(torch.full((10, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in range(2))
    piq.kv8_read(b.cache, ints(cu), ints([0] * n), b.gpu_table(), 10, BF16, out=out,
                 status=status)
    assert bool(bad) == (status.tolist()[0] == piq.PIQ_ERR_INVALID_ARG)
    for i in bad:
        assert status.tolist()[1] in bad
        for o in out:
            assert torch.isnan(o[max(cu[i], 0):max(min(cu[i + 1], 10), 0)]).all()


# ----------------------------------------------------------------------- many heads
@pytest.mark.parametrize("max_len", [40, 100000])
def test_attention_more_heads_than_a_grid_dimension(max_len):
    kvh, group, dim, n = 1024, 65, 64, 20
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = piq.kv8_cache(3, kvh, dim, 16)
    k, v = (torch.randn(n, kvh, dim, generator=g, device="cuda") for _ in range(2))
    table = ints([[2, 0]])
    piq.kv8_append(cache, k, v, ints([0, n]), ints([0]), table)
    q = torch.randn(1, kvh * group, dim, generator=g, device="cuda").to(BF16)
    out, lse = piq.kv8_attention(cache, q, ints([0, 1]), ints([n]), table, 1, max_len,
                                 return_lse=True)
    kk, vv = (x.double() for x in piq.kv8_read(cache, ints([0, n]), ints([0]), table, n, FP32))
    s = torch.einsum("hgd,nhd->hgn", q[0].view(kvh, group, dim).double(), kk) * dim ** -0.5
    p = torch.softmax(s, 2)
    ref = torch.einsum("hgn,nhd->hgd", p, vv).view(1, -1, dim)
    size = torch.einsum("hgn,nhd->hgd", p, vv.abs()).view(1, -1, dim)
    # the roundings of the weights (2^-11 each) and of the result; the scores' (d + 4) 2^-23 of
    # their sums of magnitudes, which are below 2^7 here, twice, and the exponential's 2^-20
    off = 2 * (dim + 4) * 2.0 ** -23 * 2 ** 7 + 2.0 ** -20
    tol = size * (2.0 ** -11 + 2 * off) + ref.abs() * half_step(BF16) * 1.01 + 2.0 ** -25
    assert ((out.double() - ref).abs() <= tol).all()
    assert ((lse[0].double() - torch.logsumexp(s, 2).view(-1)).abs() <= off + 2.0 ** -18).all()


def test_check_status_waits_for_every_stream():
    rng = np.random.default_rng(26)
    b = Batch(rng, [40], 2, 64, 16, BF16)
    b.append([20])
    status, kv = piq.new_status(), rand(rng, (1, 2, 64), BF16)
    cu, lens, table = ints([0, 1]), ints([20]), b.gpu_table().clone()
    table[0, 1] = 10 ** 6
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)            # some 30 ms ahead of the call
        piq.kv8_append(b.cache, kv, kv, cu, lens, table, stream=side, status=status)
        with pytest.raises(piq.PiqError):
            piq.check_status(status)
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0]
