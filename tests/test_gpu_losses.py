"""The preference and policy losses on logits against their formulas in 64 bits.

Tolerances.  A row's sum of exponentials: each term has 2^-22 from the exponential and |z - max| log2(e) 2^-23 from its
argument (5e-6 at 30), the sum up to 140 sequential fp32 additions (8e-6): logp is within 2e-5 absolutely.  A softmax
value has the same relative error twice (argument and sum): 5e-5 in the norm of an fp32 gradient; a bf16 one is rounded
by up to 2^-8 of each value (4e-3 in the norm, reached where one value dominates).  A pair's margin sums n rows: n 2e-5, and the coefficient of its gradient changes
by at most beta times that relatively.
"""
import math

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402

LOGP = 2e-5


def inputs(rows, vocab, dtype, seed=0, ignored=0.2, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn(rows, ld or vocab, device="cuda", generator=g) * 3).to(dtype)[:, :vocab]
    y = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    z[torch.arange(rows), y] += 6
    y = torch.where(torch.rand(rows, device="cuda", generator=g) < ignored, torch.full_like(y, -100), y)
    noise = torch.randn(4, rows, device="cuda", generator=g)
    return z, y, noise


def log_probs(z, y):
    x = torch.log_softmax(z.double().cpu(), 1)
    y = y.cpu()
    counts = (y >= 0) & (y < z.shape[1])
    at = torch.where(counts, y, 0)
    return x, torch.where(counts, x[torch.arange(len(y)), at], 0.0), counts, at


def gradient(x, at, c):
    d = -torch.exp(x) * c[:, None]
    d[torch.arange(len(c)), at] += c
    return torch.where(c[:, None] != 0, d, 0.0)


def near(got, ref, tol):
    n = float(ref.norm())
    e = float((got.double().cpu() - ref).norm())
    assert e <= tol * n if n else e == 0, (e, n)


def grad_tol(dtype):
    return 4e-3 if dtype == torch.bfloat16 else 5e-5


def ref_pref(z, y, pairs, ref, beta, eps, scale):
    x, logp, counts, at = log_probs(z, y)
    r = torch.zeros_like(logp) if ref is None else ref.double().cpu()
    d = torch.where(counts, logp - r, 0.0)
    margin = torch.stack([d[a:a + n].sum() - d[b:b + m].sum() for a, b, n, m in pairs]) if pairs else torch.zeros(0).double()
    h = beta * margin
    sp = torch.nn.functional.softplus
    loss = scale * ((1 - eps) * sp(-h) + eps * sp(h)).sum()
    dh = scale * beta * (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h))
    c = torch.zeros_like(logp)
    for (a, b, n, m), v in zip(pairs, dh):
        c[a:a + n], c[b:b + m] = v, -v
    c = torch.where(counts, c, 0.0)
    return loss, logp, margin, gradient(x, at, c)


def check_pref(z, y, pairs, ref, beta=0.3, eps=0.1, scale=0.5, **kw):
    want = ref_pref(z.clone(), y, pairs, ref, beta, eps, scale)
    loss, logp, margin, dz = api.pref_loss(z, y, pairs, ref, beta=beta, label_smoothing=eps, scale=scale, **kw)
    rows = max([n + m for _, _, n, m in pairs], default=0)
    assert float((logp.double().cpu() - want[1]).abs().max()) <= LOGP
    if pairs:
        # an fp32 margin is rounded to 2^-24 of its size
        assert bool(((margin.double().cpu() - want[2]).abs() <= LOGP * rows + 1e-7 * want[2].abs()).all())
    assert abs(float(loss) - float(want[0])) <= scale * beta * LOGP * rows * len(pairs) + 1e-6 * abs(float(want[0]))
    near(dz, want[3], grad_tol(z.dtype) + beta * LOGP * rows)
    return loss, logp, margin, dz


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 1000, 4095, 4096, 4097, 50021])
def test_preference_vocab_sizes(vocab, dtype):
    z, y, noise = inputs(23, vocab, dtype, seed=vocab)
    check_pref(z, y, [(0, 5, 5, 6), (12, 15, 3, 1)], noise[0] * 0.3 - 5)


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 262144), (torch.float32, 262144), (torch.bfloat16, 131073),
                                         (torch.float32, 70001)])
def test_longest_rows(dtype, vocab):
    z, y, noise = inputs(6, vocab, dtype, seed=1)
    check_pref(z, y, [(0, 3, 3, 3)], noise[0])
    check_policy(z, y, noise)


def test_preference_tables():
    """Empty responses, pairs in any order, rows of no pair, no reference, no pair, many pairs."""
    z, y, noise = inputs(60, 321, torch.float32, seed=2)
    check_pref(z, y, [(40, 0, 10, 5), (20, 30, 0, 7), (6, 55, 3, 5)], None)
    check_pref(z, y, [(0, 0, 0, 0)], noise[0])
    loss, logp, margin, dz = check_pref(z, y, [], noise[0])
    assert float(loss) == 0 and not dz.count_nonzero() and margin.numel() == 0
    z, y, noise = inputs(700, 64, torch.bfloat16, seed=3)
    check_pref(z, y, [(7 * i, 7 * i + 3, 3, 4) for i in range(100)], noise[0])


def test_preference_far_margins():
    """Margins of hundreds, either way: the loss is |h| or 0 and nothing overflows."""
    z, y, noise = inputs(80, 50, torch.float32, seed=4, ignored=0.0)
    z = z * 10
    for eps in (0.0, 0.2):
        for ref in (torch.full((80,), 30.0, device="cuda"), torch.full((80,), -30.0, device="cuda")):
            ref[40:] *= -1
            check_pref(z, y, [(0, 40, 40, 40)], ref, beta=1.0, eps=eps)


def ref_policy(z, y, old, adv, ref, lo, hi, kl, scale):
    x, logp, counts, at = log_probs(z, y)
    old, adv = old.double().cpu(), adv.double().cpu()
    r = torch.exp(logp - old)
    ra, ca = r * adv, r.clamp(1 - lo, 1 + hi) * adv
    loss, c = -torch.minimum(ra, ca), torch.where(ra <= ca, -ra, 0.0)
    if kl:
        e = ref.double().cpu() - logp
        loss, c = loss + kl * (torch.exp(e) - e - 1), c - kl * torch.expm1(e)
    c = torch.where(counts, scale * c, 0.0)
    return scale * loss[counts].sum(), logp, gradient(x, at, c), scale * loss[counts].abs().sum()


def check_policy(z, y, noise, kl=0.05, lo=0.2, hi=0.3, scale=0.1, **kw):
    logp = log_probs(z, y)[1].float().cuda()
    ratio = noise[1] * 0.3
    for end in (math.log(1 - lo), math.log(1 + hi)):     # off the kinks of the clip by more than logp's error
        ratio = torch.where((ratio - end).abs() < 1e-3, end + 2e-3, ratio)
    old, adv, ref = logp - ratio, noise[2].contiguous(), (logp + noise[3] * 0.5).contiguous()
    want = ref_policy(z.clone(), y, old, adv, ref, lo, hi, kl, scale)
    got = api.policy_loss(z, y, old, adv, ref if kl else None, clip_low=lo, clip_high=hi, kl_coef=kl, scale=scale, **kw)
    assert float((got[1].double().cpu() - want[1]).abs().max()) <= LOGP
    # d loss / d logp is at most (r |A| + kl e^x) <= a few times |loss| terms: logp's error times that
    assert abs(float(got[0]) - float(want[0])) <= 10 * LOGP * float(want[3]) + 1e-7
    near(got[2], want[2], grad_tol(z.dtype) + 5 * LOGP)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 5), (1, 40000), (3, 1001), (37, 4099), (300, 8192), (2, 131072)])
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_policy(rows, vocab, dtype, kl):
    z, y, noise = inputs(rows, vocab, dtype, seed=rows + vocab, ignored=0.2 if rows > 1 else 0.0)
    check_policy(z, y, noise, kl=kl)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_slices_and_in_place(dtype):
    z, y, noise = inputs(20, 1003, dtype, seed=5, ld=1009)           # padded, odd rows
    a = check_policy(z, y, noise)
    z1, y1 = z[1:], y[1:]                                            # the usual shift: bases off any boundary
    b = check_policy(z1, y1.contiguous(), noise[:, 1:])
    check_pref(z1, y[1:], [(0, 9, 9, 9)], noise[0, 1:])
    out = torch.zeros(20, 1024, dtype=dtype, device="cuda")[:, 3:1006]   # gradient rows lie otherwise than logits rows
    c = check_policy(z, y, noise, dlogits=out)
    assert torch.equal(a[2], c[2])
    for f in (check_policy, None):
        x = torch.zeros(20, 1009, dtype=dtype, device="cuda")[:, :1003].copy_(z)      # z's own layout: the same bits
        if f:
            d = check_policy(x, y, noise, dlogits=x)
            assert torch.equal(d[2], a[2]) and d[2].data_ptr() == x.data_ptr()
        else:
            want = api.pref_loss(z, y, [(0, 9, 9, 9)], noise[0])
            got = api.pref_loss(x, y, [(0, 9, 9, 9)], noise[0], dlogits=x)
            assert all(torch.equal(p, q) for p, q in zip(want, got))
    assert b is not None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_logits(dtype):
    """Logits of -inf and of the type's lowest value, all of a thread's and all but the label's; NaN and infinity in
    rows that do not count; labels past the vocabulary."""
    z, y, noise = inputs(12, 5000, dtype, seed=6, ignored=0.0)
    low = torch.finfo(dtype).min
    keep = torch.arange(5000, device="cuda") % 3 == 0
    keep[y] = True
    z[0:3, ~keep] = -math.inf
    z[3:6, ~keep] = low
    z[6, :] = -math.inf
    z[6, y[6]] = 1.0
    z[7, :] = math.nan
    z[8, 17] = math.inf
    y[7], y[8] = -1, 5000
    got = check_policy(z, y, noise)
    assert float(got[1][6]) == 0.0 and not got[2][7].count_nonzero() and not got[2][8].count_nonzero()
    got = check_pref(z, y, [(0, 6, 6, 6)], noise[0])
    assert not got[3][7].count_nonzero()
    y[7] = 3
    assert math.isnan(float(api.policy_loss(z, y, noise[0], noise[1])[0]))


def test_no_row_counts_and_no_rows():
    z, y, noise = inputs(9, 100, torch.bfloat16, seed=7)
    y[:] = -100
    loss, logp, dz = api.policy_loss(z, y, noise[0], noise[1])
    assert float(loss) == 0 and not logp.count_nonzero() and not dz.count_nonzero()
    loss, logp, margin, dz = api.pref_loss(z, y, [(0, 4, 4, 4)], noise[0], beta=1.0)
    assert abs(float(loss) - math.log(2)) < 1e-6 and float(margin[0]) == 0 and not dz.count_nonzero()
    e = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(0, device="cuda")
    loss, logp, dz = api.policy_loss(e, f.long(), f, f)
    assert float(loss) == 0 and dz.shape == (0, 100)
    assert float(api.pref_loss(e, f.long(), [])[0]) == 0


def test_without_gradient_and_reference_flow():
    """logp of a call without gradient is what a later call takes as the reference: a margin of zero."""
    z, y, noise = inputs(30, 777, torch.bfloat16, seed=8)
    _, logp, _, none = api.pref_loss(z, y, [], want_grad=False)
    assert none is None
    loss, logp2, margin, _ = api.pref_loss(z, y, [(0, 15, 15, 15)], logp)
    assert torch.equal(logp, logp2) and float(margin[0]) == 0 and abs(float(loss) - math.log(2)) < 1e-6
    assert torch.equal(api.policy_loss(z, y, logp, noise[0], want_grad=False)[1], logp)


def test_gradients_against_differences():
    """Central differences in 64 bits of each loss along a random direction, step 1e-4 (truncation 1e-8)."""
    z, y, noise = inputs(16, 200, torch.float32, seed=9)
    pairs, ref = [(0, 8, 8, 8)], noise[0] - 4
    logp = log_probs(z, y)[1].float().cuda()
    old, adv, rl = logp - noise[1] * 0.05, noise[2].contiguous(), logp + noise[3]
    dirn = torch.randn(z.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    zs = [z.double().cpu() + s * dirn for s in (1e-4, -1e-4)]
    for dz, f in ((api.pref_loss(z, y, pairs, ref, beta=0.2, label_smoothing=0.1)[3],
                   lambda x: ref_pref(x, y, pairs, ref, 0.2, 0.1, 1.0)[0]),
                  (api.policy_loss(z, y, old, adv, rl, kl_coef=0.1)[2],
                   lambda x: ref_policy(x, y, old, adv, rl, 0.2, 0.2, 0.1, 1.0)[0])):
        num = float(f(zs[0]) - f(zs[1])) / 2e-4
        ana = float((dz.double().cpu() * dirn).sum())
        assert abs(num - ana) <= 1e-3 * float(dz.double().norm()) + 1e-6, (num, ana)


def test_repeated_calls_and_streams():
    z, y, noise = inputs(400, 32001, torch.bfloat16, seed=10)
    pairs = api.pref_pairs([(0, 200, 200, 200)])
    f = lambda s: api.pref_loss(z, y, pairs, noise[0], stream=s) + api.policy_loss(z, y, noise[1], noise[2], stream=s)  # noqa: E731
    first = f(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, None, side):
        again = f(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_refusals():
    z, y, noise = inputs(10, 64, torch.bfloat16, seed=11)

    def refused(status, f):
        with pytest.raises(native.LoraError) as e:
            f()
        assert e.value.status == status

    refused(8, lambda: api.pref_loss(z, y, [(0, 5, 6, 5)]))              # a row in two responses
    refused(8, lambda: api.pref_loss(z, y, [(0, 8, 4, 3)]))              # past the rows
    refused(8, lambda: api.pref_loss(z, y, [(0, -1, 4, 1)]))
    refused(8, lambda: api.pref_loss(z, y, [(0, 0, 0, 0)] * 1025))
    refused(1, lambda: api.pref_loss(z, y, [], beta=math.nan))
    refused(1, lambda: api.pref_loss(z, y, [], label_smoothing=1.5))
    refused(1, lambda: api.policy_loss(z, y, noise[0], noise[1], clip_low=-0.1))
    refused(1, lambda: api.policy_loss(z, y, noise[0], noise[1], clip_high=math.inf))
    refused(1, lambda: api.policy_loss(z, y, noise[0], noise[1], kl_coef=0.1))   # a KL term without a reference
    refused(3, lambda: api.policy_loss(torch.zeros(1, 262145, dtype=torch.bfloat16, device="cuda"), y[:1], noise[0, :1], noise[1, :1]))
    refused(6, lambda: api.policy_loss(z, y, noise[0], noise[1], ws=torch.zeros(64, dtype=torch.uint8, device="cuda")))
    with pytest.raises(TypeError):
        api.policy_loss(z.half(), y, noise[0], noise[1])
    with pytest.raises(ValueError):
        api.policy_loss(z, y.int(), noise[0], noise[1])
    with pytest.raises(ValueError):
        api.policy_loss(z, y, noise[0, :5], noise[1])
    with pytest.raises(ValueError):
        api.pref_loss(z, y, [(0, 1, 2)])


@pytest.mark.parametrize("vocab", [1000, 30001])
def test_offsets_past_32_bits(vocab):
    """Rows far apart: element offsets past 2^32, of the logits and of their gradient."""
    rows, ld, n = 4500, 2 ** 20, 6
    assert (rows - n) * ld > 2 ** 32
    z0, y0, noise = inputs(n, vocab, torch.bfloat16, seed=21, ignored=0.0)
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")     # 9.4 GB, only the last rows are filled
    z = buf[:, :vocab]
    z[rows - n:] = z0
    y = torch.full((rows,), -1, device="cuda")
    y[rows - n:] = y0
    ref = torch.zeros(rows, device="cuda")
    ref[rows - n:] = noise[0, :n]
    pairs, near_pairs = [(rows - n, rows - n + 3, 3, 3)], [(0, 3, 3, 3)]
    want = api.pref_loss(z0.clone(), y0, near_pairs, noise[0, :n].contiguous())
    dz = buf[:, 2 ** 19:2 ** 19 + vocab]
    got = api.pref_loss(z, y, pairs, ref, dlogits=dz)
    assert torch.allclose(got[0], want[0], rtol=1e-5) and torch.allclose(got[2], want[2], rtol=1e-4, atol=n * LOGP)
    assert torch.allclose(got[1][rows - n:], want[1], atol=LOGP) and not got[1][:rows - n].count_nonzero()
    near(dz[rows - n:], want[3].double().cpu(), grad_tol(torch.bfloat16))
    assert not dz[:rows - n].count_nonzero()
    old, adv = ref - 0.1, ref + 1
    want = api.policy_loss(z0.clone(), y0, old[rows - n:].contiguous(), adv[rows - n:].contiguous())
    got = api.policy_loss(z, y, old, adv, dlogits=z)                     # in place
    assert torch.allclose(got[0], want[0], rtol=1e-4)
    near(z[rows - n:], want[2].double().cpu(), grad_tol(torch.bfloat16))


@pytest.mark.parametrize("n_pairs,rows", [(0, 9), (1, 300), (19, 200), (64, 200), (65, 200), (300, 700)])
def test_long_rows_with_few_and_many_pairs(n_pairs, rows):
    """Rows of a vocabulary beyond a CTA's registers: the pairs by the pass over the logits, or by a kernel of their own."""
    z, y, noise = inputs(rows, 20001, torch.bfloat16, seed=n_pairs)
    each = rows // max(1, 2 * n_pairs)
    pairs = [(2 * i * each, (2 * i + 1) * each, each, each - (i % 2 if each > 1 else 0)) for i in range(n_pairs)]
    first = check_pref(z, y, pairs, noise[0].contiguous())
    again = check_pref(z, y, pairs, noise[0].contiguous())
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("vocab,n_pairs", [(300, 3), (20001, 3), (20001, 70)])
def test_labels_of_probability_zero(vocab, n_pairs):
    """A label outside a restricted vocabulary has log p = -inf and its pair an infinite margin.  The loss is that of the limit:
    a term whose weight is zero (no smoothing, or nothing but it) counts nothing, however large; nothing becomes NaN."""
    z, y, noise = inputs(4 * n_pairs, vocab, torch.float32, seed=vocab, ignored=0.0)
    pairs = [(4 * i, 4 * i + 2, 2, 2) for i in range(n_pairs)]
    for side, sign in ((0, -1.0), (2, 1.0)):
        x = z.clone()
        x[4 + side, y[4 + side]] = -math.inf          # of the second pair
        for eps in (0.0, 1.0, 0.25):
            loss, logp, margin, dz = api.pref_loss(x, y, pairs, noise[0].contiguous(), beta=0.3, label_smoothing=eps)
            assert float(margin[1]) == sign * math.inf and float(logp[4 + side]) == -math.inf
            assert torch.isfinite(dz).all()
            h = 0.3 * torch.cat([margin[:1], margin[2:]]).double().cpu()
            sp = torch.nn.functional.softplus
            rest = float(((1 - eps) * sp(-h) + eps * sp(h)).sum())
            weight = eps if side else 1 - eps            # of the term that grows
            if weight:
                assert float(loss) == math.inf
            else:
                assert abs(float(loss) - rest) <= 1e-5 * rest + 1e-6
                assert not dz[4:8].count_nonzero()


@pytest.mark.parametrize("n_pairs,each,own", [(0, 0, 0), (1, 64, 0), (16, 64, 0), (16, 1, 0), (17, 5, 1), (1, 65, 1), (2, 700, 1),
                                              (64, 3, 1)])
def test_who_forms_the_pairs_of_long_rows(n_pairs, each, own):
    """Few short pairs are formed by the pass over the logits, others by a kernel with a CTA a pair: a long pair is not left
    to one warp.  The results are right either way."""
    z, y, noise = inputs(max(2 * n_pairs * each, 5), 17000, torch.bfloat16, seed=n_pairs + each)
    pairs = [(2 * i * each, (2 * i + 1) * each, each, each) for i in range(n_pairs)]
    native.timing_begin()
    got = check_pref(z, y, pairs, noise[0] * 0.3 - 5)
    torch.cuda.synchronize()
    launches = native.timing_end()
    assert launches["loss_rows"][1] == 1 and launches.get("loss_pairs", (0, 0))[1] == own
    again = api.pref_loss(z, y, pairs, noise[0] * 0.3 - 5, beta=0.3, label_smoothing=0.1, scale=0.5)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,ld", [(1003, 1003), (1003, 1009), (20001, 20001), (64, 64)])
def test_gradients_lie_like_the_logits(vocab, ld, dtype):
    """The gradient that a call allocates has the logits' strides and their place in a 16-byte vector, wherever a slice starts:
    else it would be stored element by element."""
    z, y, noise = inputs(20, vocab, dtype, seed=vocab, ld=ld)
    for first in (0, 1, 3):
        x, labels, n = z[first:], y[first:].contiguous(), noise[:, first:]
        for dz in (check_policy(x, labels, n)[2], check_pref(x, labels, [(0, 8, 8, 8)], n[0].contiguous())[3]):
            assert dz.stride() == x.stride() and dz.data_ptr() % 16 == x.data_ptr() % 16
            assert dz.is_contiguous() == x.is_contiguous()
    one = z[5:6]
    assert check_policy(one, y[5:6].clamp(min=0).contiguous(), noise[:, 5:6])[2].shape == (1, vocab)
