"""Causal attention over packed prompts, against fp64.

Tolerance, per output element, from the arithmetic (e = eps of the 16-bit type, so a rounding is off by
e / 2 of the value):
  * the final rounding: e / 2 |o|;
  * the weights are rounded to the type before the product with V: e / 2 of sum_j w_j |v_j|, w the
    softmax (their sum is taken before the rounding); fp16 weights below 2^-14 are off by up to 2^-25, n of
    them, against a sum of at least 1: n 2^-25 max |v|;
  * a score is an fp32 sum of d exact products, off by at most (d + 2) 2^-24 sum |q_c k_c|, and a base change
    off by 2^-23 of it, in the exponent; exp2 off by 2^-22; fp32 sums over n keys by n 2^-24: each times
    max |v|, twice (numerator and sum).
"""
import numpy as np
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev

pytestmark = pytest.mark.gpu

EPS = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def cu_of(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def make(lens, nh, nkv, d, dtype, seed=0, spare=0, pad=0, qscale=2.0):
    """q, k, v as columns of one QKV tensor (pad columns before them); rows behind the last sequence hold NaN."""
    T = sum(lens)
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn((T + spare, pad + (nh + 2 * nkv) * d), generator=g, device=dev())
    x[:, pad:pad + nh * d] *= qscale
    x = x.to(TDT[dtype])
    x[T:] = float("nan")
    a, b = pad + nh * d, pad + (nh + nkv) * d
    return x[:, pad:a], x[:, a:b], x[:, b:b + nkv * d]


def check_rows(got, q, k, v, cu, nh, nkv, d, scale=None, seqs=None, heads=None):
    scale = d ** -0.5 if scale is None else scale
    e = EPS[q.dtype]
    for b in seqs if seqs is not None else range(len(cu) - 1):
        a, z = cu[b], cu[b + 1]
        n = z - a
        if n == 0:
            continue
        hide = torch.ones((n, n), dtype=torch.bool, device=dev()).triu(1)
        for h in heads if heads is not None else range(nh):
            c, kc = slice(h * d, (h + 1) * d), slice(h // (nh // nkv) * d, (h // (nh // nkv) + 1) * d)
            Q, K, V = q[a:z, c].double(), k[a:z, kc].double(), v[a:z, kc].double()
            s = (Q @ K.T * scale).masked_fill(hide, float("-inf"))
            w = torch.softmax(s, 1)
            ref = w @ V
            mag = (Q.abs() @ K.abs().T * scale).masked_fill(hide, 0).amax(1, keepdim=True)
            big = s.masked_fill(hide, 0).abs().amax(1, keepdim=True)
            vmax = V.abs().max()
            ds = (d + 2) * 2.0 ** -24 * mag + 2.0 ** -23 * big
            limit = e / 2 * ref.abs() + e / 2 * (1 + e) * (w @ V.abs()) + vmax * (
                2 * ds + 2 * (2.0 ** -22 + n * 2.0 ** -24) + n * 2.0 ** -25) + 2.0 ** -25
            o = got[a:z, c].double()
            assert torch.isfinite(o).all(), (b, h, n)
            off = (o - ref).abs()
            assert (off <= limit).all(), (b, h, n, float((off / limit).max()))


def run(lens, nh, nkv, d, dtype, seed=0, spare=0, pad=0, max_len=None, scale=None, **kw):
    q, k, v = make(lens, nh, nkv, d, dtype, seed, spare, pad)
    cu = cu_of(lens)
    err = rpp.new_error_word()
    out = torch.full((q.shape[0], nh * d), 7.0, dtype=q.dtype, device=dev())
    rpp.attention_causal_varlen(q, k, v, ints(cu), len(lens), max_len or max(lens), nh, nkv, d, scale=scale, out=out,
                                err=err)
    assert rpp.get_device_error(err) == 0
    check_rows(out, q, k, v, cu, nh, nkv, d, scale, **kw)
    assert (out[cu[-1]:] == 7).all()          # rows behind the last sequence stay as they were


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 17, 127, 128])
def test_one_tile(dtype, d, n):
    run([n], 2, 2, d, dtype, seed=n, spare=3)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [129, 255, 256, 257, 383, 384, 385, 511, 513, 640, 1000, 1025])
def test_tiles(dtype, d, n):
    run([n], 3, 1, d, dtype, seed=n, spare=1)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(1, 1), (8, 2), (12, 12), (5, 1), (6, 3), (32, 8)])
def test_ragged_batches(dtype, d, nh, nkv):
    run([1, 0, 300, 128, 5, 129, 0, 256, 77, 257, 640, 2, 0], nh, nkv, d, dtype, seed=nh, spare=50, pad=8)


@pytest.mark.parametrize("d,max_len", [(64, 128), (128, 128), (64, 100), (128, 2000), (64, 262144)])
def test_max_len_above_the_lengths(d, max_len):
    run([100, 3, 0, 50, 1], 4, 2, d, "bf16", max_len=max_len)


@pytest.mark.parametrize("B,hi", [(300, 12), (4096, 5), (700, 150), (64, 384)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_prompts(B, hi, d):
    lens = [int(x) for x in np.random.default_rng(B).integers(0, hi + 1, B)]
    run(lens, 2, 1, d, "bf16", seqs=list(range(0, B, max(1, B // 150))) + [B - 1])


@pytest.mark.parametrize("dtype,d,nh,nkv,lens", [("bf16", 128, 8, 2, [5000, 1, 3001]), ("fp16", 64, 4, 4, [6007]),
                                                 ("bf16", 64, 16, 1, [2500, 2500, 40])])
def test_long(dtype, d, nh, nkv, lens):
    run(lens, nh, nkv, d, dtype, heads=[0, nh - 1])


def test_scale_and_rows_apart():
    run([300, 40], 4, 2, 64, "fp16", scale=0.4, pad=24)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[600, 90], [128], [100]])
def test_scores_far_apart(d, lens):
    """Scores that climb along the keys, by far more than the lazily moved maximum allows."""
    q, k, v = make(lens, 2, 1, d, "fp16")
    T = sum(lens)
    k.zero_()
    k[:, 0] = torch.linspace(-200, 200, T, device=dev()).half()
    q.zero_()
    q[:, ::d] = 4.0
    err = rpp.new_error_word()
    out = rpp.attention_causal_varlen(q, k, v, ints(cu_of(lens)), len(lens), max(lens), 2, 1, d, err=err)
    assert rpp.get_device_error(err) == 0
    check_rows(out, q, k, v, cu_of(lens), 2, 1, d)

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh", [1, 2])
def test_many_weights_far_below_the_maximum(d, nh):
    """65536 fp16 keys, the first 26 powers of two above the others in weight: in the last rows those are
    2^-10 of the sum, and the output is theirs (the first value is 0, theirs 1).

    Tolerance: two roundings, of the weights and of the output, 2^-11 each; weights of up to 2^8 are
    kept 2^7 times as large, so what is below fp16's smallest step, 2^-24, is half a step of 2^-7
    of it off: i 2^-32 in row i; fp32 sums of i like terms, i 2^-24 of each of numerator and denominator;
    2^-16 for the exponent, 26 2^-23 off; half a step of the smallest fp16 outputs."""
    n = 65536
    q, k, v = (torch.zeros(n, w * d, device=dev(), dtype=torch.float16) for w in (nh, 1, 1))
    q[:, ::d] = 8.0
    k[0, 0] = 18.02                                                 # score 8 * 18.02 / 8, e^-18.02 = 2^-26
    v[1:] = 1
    err = rpp.new_error_word()
    got = rpp.attention_causal_varlen(q, k, v, ints([0, n]), 1, n, nh, 1, d, scale=0.125, err=err).double()
    assert rpp.get_device_error(err) == 0
    i = torch.arange(n, device=dev(), dtype=torch.float64)[:, None]
    w = torch.exp(-k[0, 0].double()) * i
    ref = w / (1 + w)
    limit = ref * (2 * 2.0 ** -11 + 2 * i * 2.0 ** -24 + 2.0 ** -16) + i * 2.0 ** -32 + 2.0 ** -25
    worst = ((got - ref).abs() - limit).argmax().item() // got.shape[1]
    assert ((got - ref).abs() <= limit).all(), (worst, float(got[worst, 0]), float(ref[worst]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh", [1, 2])
def test_weights_as_large_as_the_lazy_maximum_lets_them_be(d, nh):
    """fp16 scores whose maximum climbs by 7.9 powers of two after the first tile, too little to move it."""
    lens = [700, 130]
    q, k, v = make(lens, nh, 1, d, "fp16")
    q.zero_()
    q[:, ::d] = 8.0
    k.zero_()
    for a, n in ((0, 700), (700, 130)):
        k[a + 128:a + n, 0] = 5.475                                 # e^5.475 = 2^7.9
    cu = cu_of(lens)
    out = rpp.attention_causal_varlen(q, k, v, ints(cu), 2, 700, nh, 1, d, scale=0.125)
    check_rows(out, q, k, v, cu, nh, 1, d, 0.125)



@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,where", [([300, 200], [5, 127, 128, 130, 255, 256, 299]), ([100, 28], [0, 50, 99]),
                                        ([513], [256, 383, 384, 511, 512])])
@pytest.mark.parametrize("what", ["k", "v"])
def test_what_a_row_must_not_see_stays_out(d, lens, where, what):
    """NaN and infinities in one key or value row: rows before it, and other sequences, as without it; rows
    from it on as the formula has them."""
    q, k, v = make(lens, 2, 1, d, "bf16")
    cu = cu_of(lens)
    base = rpp.attention_causal_varlen(q, k, v, ints(cu), len(lens), max(lens), 2, 1, d)
    for j in where:
        for bad in (float("nan"), float("inf"), float("-inf")):
            k2, v2 = k.clone(), v.clone()
            (k2 if what == "k" else v2)[j, 3] = bad
            err = rpp.new_error_word()
            out = rpp.attention_causal_varlen(q, k2, v2, ints(cu), len(lens), max(lens), 2, 1, d, err=err)
            assert rpp.get_device_error(err) == 0
            assert torch.equal(out[:j], base[:j])
            assert torch.equal(out[lens[0]:], base[lens[0]:])
            if what == "v":
                seen = out[j:lens[0]].float()
                for h in range(2):
                    col = seen[:, h * d + 3]
                    assert (torch.isnan(col) if bad != bad else col == bad).all()
                    keep = torch.ones(2 * d, dtype=torch.bool, device=dev())
                    keep[[3, d + 3]] = False
                    assert torch.isfinite(seen[:, keep]).all()


def test_the_same_result_every_time():
    lens = [int(x) for x in np.random.default_rng(1).integers(1, 900, 40)]
    q, k, v = make(lens, 8, 2, 128, "bf16")
    a = (q, k, v, ints(cu_of(lens)), len(lens), 900, 8, 2, 128)
    first = rpp.attention_causal_varlen(*a)
    for _ in range(5):
        assert torch.equal(first, rpp.attention_causal_varlen(*a))


def test_device_errors():
    q, k, v = make([100, 28], 2, 1, 64, "bf16")
    for cu, max_len, code in (([0, 100, 129], 128, rpp.RPP_DERR_ROWS), ([0, 100, 128], 99, rpp.RPP_DERR_LENGTH),
                              ([0, 100, 50], 128, rpp.RPP_DERR_ROWS), ([-4, 100, 128], 128, rpp.RPP_DERR_ROWS)):
        err = rpp.new_error_word()
        out = torch.full((128, 128), 7.0, dtype=torch.bfloat16, device=dev())
        rpp.attention_causal_varlen(q, k, v, ints(cu), 2, max_len, 2, 1, 64, out=out, err=err)
        assert rpp.get_device_error(err) == code
        assert (out == 7).all()
    err.fill_(42)
    rpp.attention_causal_varlen(q, k, v, ints([0, 100, 128]), 2, 128, 2, 1, 64, out=out, err=err)
    assert (out == 7).all() and rpp.get_device_error(err) == 42


def test_after_other_tensor_memory_users():
    """Tensor memory keeps what the kernel before left (NaN here): it must not reach an output."""
    q, k, v = make([700, 3], 2, 1, 128, "bf16")
    bad = torch.full_like(q, float("nan"))
    for _ in range(3):
        rpp.attention_causal_varlen(bad, k, v, ints([0, 700, 703]), 2, 700, 2, 1, 128)
        run([130, 1, 300], 4, 2, 128, "bf16")
        run([130, 1, 300], 4, 2, 64, "bf16")


def test_captured_and_replayed_with_other_lengths():
    nh, nkv, d, T = 4, 2, 64, 1200
    q, k, v = make([T], nh, nkv, d, "bf16")
    cu = ints([0, T, T, T])
    err = rpp.new_error_word()
    out = torch.empty(T, nh * d, dtype=torch.bfloat16, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rpp.attention_causal_varlen(q, k, v, cu, 3, T, nh, nkv, d, out=out, err=err)
    torch.cuda.synchronize()
    for lens in ([1200, 0, 0], [0, 0, 0], [1, 600, 599], [128, 128, 128], [5, 0, 1000]):
        cu.copy_(ints(cu_of(lens)))
        out.fill_(7)
        g.replay()
        assert rpp.get_device_error(err) == 0
        check_rows(out, q, k, v, cu_of(lens), nh, nkv, d)
        assert (out[sum(lens):] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_q_k_and_v_as_tensors_of_their_own(d):
    """Three tensors (three tensor maps), and K and V in the order V, K inside one."""
    lens, nh, nkv = [300, 1, 130], 4, 2
    q, k, v = make(lens, nh, nkv, d, "bf16")
    kv = torch.cat([v, k], 1)
    want = rpp.attention_causal_varlen(q, k, v, ints(cu_of(lens)), 3, 300, nh, nkv, d)
    check_rows(want, q, k, v, cu_of(lens), nh, nkv, d)
    for a in ((q.contiguous(), k.contiguous(), v.contiguous()), (q, kv[:, nkv * d:], kv[:, :nkv * d]),
              (q.contiguous(), kv[:, nkv * d:], kv[:, :nkv * d])):
        assert torch.equal(rpp.attention_causal_varlen(*a, ints(cu_of(lens)), 3, 300, nh, nkv, d), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_batch_many_times(dtype, d):
    """Items whose last queries do not exist next to full ones, several to a CTA, one launch after the other: every
    run the same, and right.  (Warps without queries run ahead of the others here.)"""
    lens, nh, nkv = [1, 0, 300, 128, 5, 129, 0, 256, 77, 257, 640, 2, 0] * 3, 32, 8
    q, k, v = make(lens, nh, nkv, d, dtype, seed=32)
    cu, err = cu_of(lens), rpp.new_error_word()
    outs = [rpp.attention_causal_varlen(q, k, v, ints(cu), len(lens), 640, nh, nkv, d, err=err) for _ in range(40)]
    assert rpp.get_device_error(err) == 0
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    check_rows(outs[0], q, k, v, cu, nh, nkv, d, seqs=range(13), heads=[0, 13, 31])


def test_two_streams_at_once():
    """Pairs of heads, single streams and both head sizes side by side: CTAs of different calls share an SM and
    its tensor memory."""
    cases = [(64, 4, 2, [300, 1, 900, 128]), (64, 3, 3, [700, 40, 1]), (128, 8, 2, [1500, 3]), (128, 5, 5, [260, 800])]
    jobs = []
    for i, (d, nh, nkv, lens) in enumerate(cases):
        jobs.append((make(lens, nh, nkv, d, "bf16", seed=i), cu_of(lens), ints(cu_of(lens)), rpp.new_error_word(),
                     torch.cuda.Stream(), [], (nh, nkv, d)))
    torch.cuda.synchronize()
    for _ in range(10):
        for (q, k, v), cu, dcu, err, s, got, (nh, nkv, d) in jobs:
            with torch.cuda.stream(s):
                got.append(rpp.attention_causal_varlen(q, k, v, dcu, len(cu) - 1, 1500, nh, nkv, d, err=err))
    torch.cuda.synchronize()
    for (q, k, v), cu, _, err, _, got, (nh, nkv, d) in jobs:
        assert rpp.get_device_error(err) == 0
        check_rows(got[0], q, k, v, cu, nh, nkv, d)
        assert all(torch.equal(got[0], g) for g in got)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,dtype,far", [(1, "fp16", 30.0), (2, "fp16", 130.0), (1, "bf16", 130.0), (2, "bf16", 60.0)])
def test_an_infinite_value_of_a_small_weight(d, nh, dtype, far):
    """A value before the diagonal tile (and in it) whose weight e^-far is above 0 whatever the arithmetic
    makes of it: the rows that see it answer the infinity, those that see both infinities NaN.  A score
    of -inf makes the weight 0, and 0 times infinity is NaN."""
    lens = [500, 300]
    q, k, v = make(lens, nh, 1, d, dtype, seed=3)
    q.zero_()
    q[:, ::d] = 8.0
    k.zero_()
    k[5, 0] = k[9, 0] = k[390, 0] = -far
    a = (ints(cu_of(lens)), 2, 500, nh, 1, d)
    err = rpp.new_error_word()
    base = rpp.attention_causal_varlen(q, k, v, *a, scale=0.125, err=err)
    assert torch.isfinite(base.float()).all()
    inf = float("inf")
    v[5, 3] = inf
    v[9, 4] = -inf
    v[5, 6] = inf
    v[9, 6] = -inf
    v[390, 8] = inf
    got = rpp.attention_causal_varlen(q, k, v, *a, scale=0.125, err=err)
    k[5, 0] = -inf
    k[390, 0] = -inf
    dropped = rpp.attention_causal_varlen(q, k, v, *a, scale=0.125, err=err)
    assert rpp.get_device_error(err) == 0

    def same(x, y):
        return ((x == y) | (torch.isnan(x) & torch.isnan(y))).all()

    for h in range(nh):
        want = base[:, h * d:(h + 1) * d].clone()
        want[5:500, 3], want[9:500, 4], want[5:9, 6], want[9:500, 6], want[390:500, 8] = inf, -inf, inf, float("nan"), inf
        x = got[:, h * d:(h + 1) * d]
        assert same(x[:, [3, 4, 6, 8]], want[:, [3, 4, 6, 8]])
        keep = [e for e in range(d) if e not in (3, 4, 6, 8)]
        assert torch.equal(x[:, keep], want[:, keep])
        x = dropped[:, h * d:(h + 1) * d]
        assert torch.isnan(x[5:500, 3]).all() and torch.isnan(x[390:500, 8]).all() and (x[9:500, 4] == -inf).all()
        assert torch.isfinite(x[:, keep].float()).all() and torch.equal(x[500:], want[500:])


def test_a_value_that_is_not_finite_costs_its_own_rows_only():
    """One infinity in the first of 64 prompts: the others take their time as before.  (Noted for good, it
    made every later item of a CTA look through its diagonal rows: 34 times the time of the batch.)"""
    lens = [int(x) for x in np.random.default_rng(1).integers(32, 385, 64)]
    q, k, v = make(lens, 16, 16, 64, "bf16")
    a = (ints(cu_of(lens)), 64, 384, 16, 16, 64)
    out = torch.empty(q.shape[0], 16 * 64, dtype=torch.bfloat16, device=dev())

    def best():
        ts = []
        for _ in range(12):
            s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            s.record()
            for _ in range(20):
                rpp.attention_causal_varlen(q, k, v, *a, out=out)
            e.record()
            e.synchronize()
            ts.append(s.elapsed_time(e))
        return min(ts[2:])

    plain = best()
    v[0, 3] = float("inf")
    spoilt = best()
    assert (out[0:lens[0], 3] == float("inf")).all()
    assert spoilt <= 2 * plain, (spoilt, plain)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh", [1, 2])
def test_rows_whose_scores_are_no_numbers_stay_nan(d, nh):
    """A query that holds NaN, or one whose scores are all -inf, beside values that are not finite: its row is NaN, the
    rows around it have the infinity."""
    lens = [400, 60]
    q, k, v = make(lens, nh, 1, d, "bf16")
    k[:, 0] = k[:, 0].abs() + 0.5
    q[200, :] = float("nan")
    q[310, :] = 0
    q[310, ::d] = float("-inf")
    v[3, 5] = float("inf")
    v[305, 6] = float("-inf")
    out = rpp.attention_causal_varlen(q, k, v, ints(cu_of(lens)), 2, 400, nh, 1, d)
    nans = torch.isnan(out.float())
    assert nans[200].all() and nans[310].all()
    rest = [i for i in range(460) if i not in (200, 310)]
    assert not nans[rest].any()
    for h in range(nh):
        col = out[:400, h * d + 5].float()
        assert (col[[i for i in rest if 3 <= i < 400]] == float("inf")).all() and torch.isfinite(col[:3]).all()
        col = out[:400, h * d + 6].float()
        assert (col[[i for i in rest if 305 <= i < 400]] == float("-inf")).all() and torch.isfinite(col[:200]).all()


@pytest.mark.parametrize("d,nh,nkv", [(64, 2, 2), (128, 4, 2), (128, 3, 3)])
def test_values_that_are_nan_all_over(d, nh, nkv):
    """Every item of a long prompt takes its outputs from the values: no wait runs out meanwhile, and the prompts
    beside it are as without it."""
    lens = [200, 20000, 333]
    q, k, v = make(lens, nh, nkv, d, "bf16")
    a = (ints(cu_of(lens)), 3, 20000, nh, nkv, d)
    base = rpp.attention_causal_varlen(q, k, v, *a)
    v[200:20200] = float("nan")
    err = rpp.new_error_word()
    out = rpp.attention_causal_varlen(q, k, v, *a, err=err)
    assert rpp.get_device_error(err) == 0
    assert torch.isnan(out[200:20200]).all()
    assert torch.equal(out[:200], base[:200]) and torch.equal(out[20200:], base[20200:])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,nh", [(64, 2), (128, 1), (128, 2)])
def test_infinities_before_and_in_the_diagonal_tile(d, nh, dtype):
    """A row's output in a column is the sum of the infinities up to it, in whichever tiles they lie; other columns are as
    without them."""
    lens, inf = [500, 300], float("inf")
    q, k, v = make(lens, nh, 1, d, dtype, seed=4, qscale=0.5)
    a = (ints(cu_of(lens)), 2, 500, nh, 1, d)
    want = rpp.attention_causal_varlen(q, k, v, *a).clone()
    for row, col, x in ((5, 3, inf), (390, 3, -inf), (200, 4, -inf), (450, 4, -inf), (128, 5, inf), (499, 6, float("nan"))):
        v[row, col] = x
    for h in range(nh):
        w = want[:500, h * d:(h + 1) * d]
        w[5:, 3], w[390:, 3], w[200:, 4], w[128:, 5], w[499:, 6] = inf, float("nan"), -inf, inf, float("nan")
    got = rpp.attention_causal_varlen(q, k, v, *a)
    assert ((got == want) | (torch.isnan(got) & torch.isnan(want))).all()
