"""Packed causal attention against the formula in 64 bits.

Tolerances (2-norm of the difference over 2-norm of the reference, per tensor): outputs are rounded to bf16 (half a
unit in the last place, 2^-9 relative at most, about 2^-9 / sqrt(3) = 1.1e-3 in the norm); P and dS are rounded to bf16
once more before their products, another 1.1e-3 in the norm of each product (independent roundings of the terms, whose
own norm is at most that of the result where the terms do not cancel, and a few times it where they do).  5e-3 leaves a
factor of three over the two together.  lse is fp32 throughout: scores of size up to 20 with 2^-24 relative
roundings in their sums of up to 128 products, and exponents and logarithms of 2^-22: 2e-5 absolute.
"""
import math

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402

TOL = 5e-3
LSE_TOL = 2e-5


def reference(Q, K, V, seqs, scale, dO=None):
    """Sequence by sequence in 64 bits on the host.  Returns O, lse (and dQ, dK, dV)."""
    q, k, v = (x.double().cpu() for x in (Q, K, V))
    g = q.shape[1] // k.shape[1]
    O, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    dQ, dK, dV = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for qs, ql, ks, kl in seqs:
        for i in range(0, ql):
            if i + kl - ql >= 0:
                break
        else:
            continue
        rows = torch.arange(i, ql)
        hidden = torch.arange(kl)[None] > (rows + kl - ql)[:, None]
        for h in range(q.shape[1]):
            qq, kk, vv = q[qs + rows, h], k[ks:ks + kl, h // g], v[ks:ks + kl, h // g]
            S = (qq @ kk.T * scale).masked_fill(hidden, -math.inf)
            L = torch.logsumexp(S, 1)
            P = torch.exp(S - L[:, None])
            O[qs + rows, h], lse[qs + rows, h] = P @ vv, L
            if dO is not None:
                do = dO.double().cpu()[qs + rows, h]
                dP = do @ vv.T
                dS = P * (dP - (P * dP).sum(1, keepdim=True)) * scale
                dQ[qs + rows, h] = dS @ kk
                dK[ks:ks + kl, h // g] += dS.T @ qq
                dV[ks:ks + kl, h // g] += P.T @ do
    return (O, lse) if dO is None else (O, lse, dQ, dK, dV)


def off(got, ref):
    got, ref = got.double().cpu(), ref
    assert torch.isfinite(got).all()
    n = ref.norm()
    return float((got - ref).norm() / n) if n > 0 else float(got.norm())


def check(Q, K, V, seqs, scale, dO, got):
    O, lse, dQ, dK, dV = got
    r = reference(Q, K, V, seqs, scale, dO)
    assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(r[1]))
    fin = torch.isfinite(r[1])
    if fin.any():
        assert float((lse.double().cpu() - r[1])[fin].abs().max()) <= LSE_TOL
    errs = {n: off(x, y) for n, x, y in zip(("O", "dQ", "dK", "dV"), (O, dQ, dK, dV), (r[0], *r[2:]))}
    assert all(e <= TOL for e in errs.values()), errs


def inputs(tq, tk, hq, hkv, d, layout="rows", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(t, h):
        x = torch.randn(max(t, 1) * h * d, device="cuda", generator=g).bfloat16()[:t * h * d]
        return x.view(h, t, d).transpose(0, 1) if layout == "heads" else x.view(t, h, d)

    if layout == "fused":
        qkv = rand(tq, hq + 2 * hkv)
        return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], rand(tq, hq)
    return rand(tq, hq), rand(tk, hkv), rand(tk, hkv), rand(tq, hq)


def packed(lengths, pad=1):
    out, at = [], 0
    for n in lengths:
        out.append((at, n, at, n))
        at += -(-n // pad) * pad
    return out, at


def run(Q, K, V, dO, seqs, scale, **kw):
    O, lse = api.attn_fwd(Q, K, V, seqs, scale=scale, **kw)
    return (O, lse, *api.attn_bwd(dO, Q, K, V, O, lse, seqs, scale=scale, **kw))


@pytest.mark.parametrize("lengths,pad", [
    ([1], 1), ([2, 1, 3], 1), ([127], 1), ([128], 1), ([129], 1), ([64, 65, 63, 1, 200], 1), ([255, 257], 128),
    ([700], 1), ([5, 0, 130, 0, 1], 1)])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (4, 2, 128)])
def test_whole_prompts(lengths, pad, hq, hkv, d):
    seqs, rows = packed(lengths, pad)
    Q, K, V, dO = inputs(rows, rows, hq, hkv, d, seed=rows)
    check(Q, K, V, seqs, d ** -0.5, dO, run(Q, K, V, dO, seqs, None))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (6, 3), (7, 1), (8, 8), (8, 1), (28, 4), (128, 1), (12, 3)])
def test_head_groups(hq, hkv):
    seqs, rows = packed([150, 33], 1)
    Q, K, V, dO = inputs(rows, rows, hq, hkv, 64, seed=hq)
    check(Q, K, V, seqs, 0.125, dO, run(Q, K, V, dO, seqs, None))


@pytest.mark.parametrize("d", [8, 24, 40, 72, 96, 104, 120])
def test_head_widths(d):
    seqs, rows = packed([140, 61], 1)
    Q, K, V, dO = inputs(rows, rows, 4, 2, d, seed=d)
    check(Q, K, V, seqs, 0.3, dO, run(Q, K, V, dO, seqs, 0.3))


@pytest.mark.parametrize("layout", ["rows", "heads", "fused"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(layout, d):
    seqs, rows = packed([200, 100], 128)
    Q, K, V, dO = inputs(rows, rows, 4, 2, d, layout, seed=3)
    got = run(Q, K, V, dO, seqs, None)
    check(Q, K, V, seqs, d ** -0.5, dO, got)
    # gradients into strided slices of one fused buffer
    fused = torch.full((rows, 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dQ, dK, dV = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    api.attn_bwd(dO, Q, K, V, got[0], got[1], seqs, dQ=dQ, dK=dK, dV=dV)
    assert torch.equal(dQ, got[2]) and torch.equal(dK, got[3]) and torch.equal(dV, got[4])


@pytest.mark.parametrize("seqs", [
    [(0, 1, 0, 500)], [(0, 1, 0, 1), (1, 1, 1, 128), (2, 1, 129, 129), (3, 1, 258, 1000)],
    [(0, 30, 0, 300), (30, 300, 300, 30), (330, 10, 330, 0), (340, 0, 330, 40), (340, 200, 370, 129)],
    [(3, 130, 5, 257), (140, 5, 270, 5)], [(0, 300, 0, 1)]])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (4, 2, 128)])
def test_queries_and_keys_of_different_lengths(seqs, hq, hkv, d):
    tq, tk = seqs[-1][0] + seqs[-1][1] + 2, seqs[-1][2] + seqs[-1][3] + 3
    Q, K, V, dO = inputs(tq, tk, hq, hkv, d, seed=tq)
    check(Q, K, V, seqs, d ** -0.5, dO, run(Q, K, V, dO, seqs, None))


def test_no_sequence_and_no_rows():
    Q, K, V, dO = inputs(40, 50, 4, 2, 64)
    O, lse, dQ, dK, dV = run(Q, K, V, dO, [], None)
    assert not any(x.count_nonzero() for x in (O, dQ, dK, dV)) and bool((lse == -math.inf).all())
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = api.attn_fwd(e, K, V, [(0, 0, 0, 50)])
    assert O.shape == (0, 4, 64) and lse.shape == (0, 4)
    dQ, dK, dV = api.attn_bwd(e, e, K, V, O, lse, [(0, 0, 0, 50)])
    assert not dK.count_nonzero() and not dV.count_nonzero()
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = api.attn_fwd(Q, kv, kv, [(0, 40, 0, 0)])
    assert not O.count_nonzero() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -3e38])
def test_rows_beside_a_sequence_do_not_reach_it(bad):
    """Rows of no sequence, and another sequence's rows, hold infinities and NaN."""
    seqs = [(0, 100, 0, 100), (128, 70, 128, 70), (198, 130, 198, 130)]
    Q, K, V, dO = inputs(400, 400, 4, 2, 128, seed=5)
    clean = run(Q, K, V, dO, seqs, None)
    Q2, K2, V2, dO2 = (x.clone() for x in (Q, K, V, dO))
    for x in (Q2, K2, V2, dO2):
        x[100:198] = bad
        x[328:] = bad
    dirty = run(Q2, K2, V2, dO2, seqs, None)
    for a, b in zip(clean, dirty):
        for s in (slice(0, 100), slice(198, 328)):
            assert torch.equal(a[s], b[s])
        assert torch.equal(a[100:128], b[100:128]) and torch.equal(a[328:], b[328:])


def test_large_scores_and_growing_maxima():
    """Scores that grow along the keys (every tile raises the running maximum) and scores of size 1e4."""
    Q, K, V, dO = inputs(1024, 1024, 2, 1, 64, seed=7)
    grow = (K.float() * 0.05 + torch.linspace(0, 30, 1024, device="cuda")[:, None, None] / 8).bfloat16()
    ones = (Q.float() * 0.05 + 1).bfloat16()
    seqs = [(0, 1024, 0, 1024)]
    O, lse, dQ, dK, dV = run(ones, grow, V, dO, seqs, None)
    ref = reference(ones, grow, V, seqs, 0.125, dO)
    assert float((lse.double().cpu() - ref[1]).abs().max()) <= LSE_TOL
    errs = {n: off(x, y) for n, x, y in zip(("O", "dK", "dV"), (O, dK, dV), (ref[0], ref[3], ref[4]))}
    assert all(e <= TOL for e in errs.values()), errs
    # dQ = dS K: here every feature of K grows alike and dS sums to zero along the keys, so the terms cancel and the
    # rounding of each to bf16 does not; the tolerance is of the terms' size, |dS| |K|
    q, k, v, do = (x.double().cpu() for x in (ones, grow, V, dO))
    hidden = torch.ones(1024, 1024, dtype=torch.bool).triu(1)
    size = torch.zeros_like(q)
    for h in range(2):
        P = torch.softmax((q[:, h] @ k[:, 0].T * 0.125).masked_fill(hidden, -math.inf), 1)
        dP = do[:, h] @ v[:, 0].T
        size[:, h] = (P * (dP - (P * dP).sum(1, keepdim=True))).abs() @ k[:, 0].abs() * 0.125
    assert float((dQ.double().cpu() - ref[2]).norm()) <= TOL * float(size.norm())
    O, lse = api.attn_fwd((Q.float() * 100).bfloat16(), (K.float() * 100).bfloat16(), V, seqs)
    assert torch.isfinite(O).all() and torch.isfinite(lse).all()


def test_gradients_against_differences():
    """Central differences of sum(O * dO) computed in 64 bits along random directions, step 1e-3: the truncation
    error is 1e-6 of the value, so the bound is that of the kernel's bf16 gradients, 5e-3 of |gradient| |direction|
    (their error is not aligned with the direction: half of that is far more than the expected projection)."""
    seqs, rows = packed([90, 41], 1)
    Q, K, V, dO = inputs(rows, rows, 4, 2, 64, seed=11)
    _, _, dQ, dK, dV = run(Q, K, V, dO, seqs, None)
    g = torch.Generator().manual_seed(1)
    base = [x.double().cpu() for x in (Q, K, V)]
    for i, grad in enumerate((dQ, dK, dV)):
        direction = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        vals = []
        for s in (1e-3, -1e-3):
            x = list(base)
            x[i] = x[i] + s * direction
            vals.append(float((reference(*x, seqs, 0.125)[0] * dO.double().cpu()).sum()))
        num = (vals[0] - vals[1]) / 2e-3
        ana = float((grad.double().cpu() * direction).sum())
        assert abs(num - ana) <= 5e-3 * float(grad.double().norm()) * 3, (i, num, ana)


def test_repeated_calls_and_streams():
    """Bit-identical from call to call, on the default stream and on another with outputs of its own."""
    seqs, rows = packed([500, 300, 130], 128)
    Q, K, V, dO = inputs(rows, rows, 8, 2, 128, seed=13)
    first = run(Q, K, V, dO, seqs, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None, side):
        again = run(Q, K, V, dO, seqs, None, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_capture():
    seqs, rows = packed([300, 77], 1)
    table = api.attn_seqs(seqs)
    Q, K, V, dO = inputs(rows, rows, 4, 2, 64, seed=17)
    want = run(Q, K, V, dO, table, None)
    O, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    dQ, dK, dV = (torch.empty_like(x) for x in want[2:])
    ws = torch.zeros(api.attn_workspace_size(rows, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.attn_fwd(Q, K, V, table, O=O, lse=lse, ws=ws)
        api.attn_bwd(dO, Q, K, V, O, lse, table, dQ=dQ, dK=dK, dV=dV, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (O, lse, dQ, dK, dV)))
    assert api.lora_device_status(ws) == 0


def test_refusals():
    Q, K, V, dO = inputs(64, 64, 4, 2, 64)

    def refused(status, seqs=((0, 64, 0, 64),), q=Q, k=K, v=V, **kw):
        with pytest.raises(native.LoraError) as e:
            api.attn_fwd(q, k, v, list(seqs), **kw)
        assert e.value.status == status

    refused(8, [(0, 65, 0, 64)])                                   # past the rows
    refused(8, [(0, 40, 0, 40), (39, 10, 40, 10)])                 # shared row
    refused(8, [(32, 10, 0, 10), (0, 10, 10, 10)])                 # not in row order
    refused(8, [(0, -1, 0, 4)])
    refused(8, [(i, 0, 0, 0) for i in range(64)] * 17)             # too many, and out of order
    refused(1, scale=0.0)
    refused(1, scale=math.inf)
    refused(3, q=inputs(64, 64, 3, 2, 64)[0])                      # 3 query heads over 2
    refused(3, *[[(0, 64, 0, 64)]], q=inputs(64, 64, 4, 2, 136)[0], k=inputs(64, 64, 4, 2, 136)[1],
            v=inputs(64, 64, 4, 2, 136)[2])                        # head too wide
    refused(2, q=torch.zeros(64 * 256 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(64, 4, 64))   # misaligned
    refused(6, ws=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(64, 4, 66, dtype=torch.bfloat16, device="cuda")[:, :, :64]
    refused(2, q=wide)                                             # strides not a multiple of 8
    refused(3, O=torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(64, 4, 64))
    with pytest.raises(ValueError):
        api.attn_fwd(Q, K, V[:32], [(0, 64, 0, 64)])
    with pytest.raises(TypeError):
        api.attn_fwd(Q.float(), K, V, [(0, 64, 0, 64)])


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 2, 128), (6, 2, 96)])
def test_few_rows_over_many_keys(hq, hkv, d):
    """Keys split over several SMs and joined: single tokens and short continuations over long prompts, rows that see
    no key of a range or none at all, unused rows between; against the formula, and against the unsplit way (a
    workspace without the region), which rounds the same products in another order."""
    lens = [(1, 9000), (7, 5003), (20, 1), (1, 130), (13, 4), (2, 0), (1, 7777), (30, 1300)]
    seqs, q, k = [], 2, 1
    for a, b in lens:
        seqs.append((q, a, k, b))
        q, k = q + a + 3, k + b + 2
    Q, K, V, _ = inputs(q, k, hq, hkv, d, seed=hq)
    O, lse = api.attn_fwd(Q, K, V, seqs)
    r = reference(Q, K, V, seqs, d ** -0.5)
    assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(r[1]))
    fin = torch.isfinite(r[1])
    assert float((lse.double().cpu() - r[1])[fin].abs().max()) <= LSE_TOL
    assert off(O, r[0]) <= TOL
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    O2, lse2 = api.attn_fwd(Q, K, V, seqs, ws=small)
    assert off(O2, r[0]) <= TOL and float((lse2 - lse)[torch.isfinite(lse2)].abs().max()) <= LSE_TOL
    again = api.attn_fwd(Q, K, V, seqs)
    assert torch.equal(O, again[0]) and torch.equal(lse, again[1])


LONG = 6000   # keys of a few-row sequence that raises the batch's mean: dQ then runs with key tiles of 128


@pytest.mark.parametrize("lengths,pad,hq,hkv,d,layout", [
    ([1, 2, 127, 128, 129], 1, 4, 1, 64, "rows"), ([255, 0, 257, 1], 128, 4, 2, 128, "rows"), ([300], 1, 3, 1, 128, "rows"),
    ([150, 33], 1, 28, 4, 64, "rows"), ([150, 33], 1, 7, 1, 40, "heads"), ([140, 61], 1, 4, 2, 8, "rows"),
    ([140, 61], 1, 4, 2, 72, "heads"), ([140, 61], 1, 8, 8, 120, "rows"), ([40, 400], 1, 16, 1, 96, "rows")])
def test_key_tiles_of_128(lengths, pad, hq, hkv, d, layout):
    """The shapes of the tests above beside a long range of keys, and past it: both forms of the dQ pass are exact to
    the same tolerance, and a sequence's gradients do not depend on the form beyond rounding."""
    short, rows = packed(lengths, pad)
    seqs = short + [(rows + 1, 8, rows + 2, LONG)]
    Q, K, V, dO = inputs(rows + 9, rows + 2 + LONG, hq, hkv, d, layout, seed=sum(lengths))
    got = run(Q, K, V, dO, seqs, None)
    check(Q, K, V, seqs, d ** -0.5, dO, got)
    alone = run(Q, K, V, dO, short, None)
    for a, b in zip(got[2:], alone[2:]):
        for q0, n, _, _ in short:
            if n:
                assert off(a[q0:q0 + n], b[q0:q0 + n].double().cpu()) <= TOL


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_beside_a_long_sequence(bad):
    """As test_rows_beside_a_sequence_do_not_reach_it, with key tiles of 128."""
    seqs = [(0, 70, 0, 70), (100, 9, 90, LONG - 5)]
    Q, K, V, dO = inputs(120, 90 + LONG, 4, 2, 64, seed=2)
    want = run(Q, K, V, dO, seqs, None)
    for t, used in ((Q, seqs), (dO, seqs)):
        mask = torch.ones(t.shape[0], dtype=torch.bool, device="cuda")
        for q0, n, _, _ in used:
            mask[q0:q0 + n] = False
        t[mask] = bad
    for t in (K, V):
        mask = torch.ones(t.shape[0], dtype=torch.bool, device="cuda")
        for _, _, k0, n in seqs:
            mask[k0:k0 + n] = False
        t[mask] = bad
    for a, b in zip(run(Q, K, V, dO, seqs, None), want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31 and 2^32: the last rows of long buffers with wide rows, every operand and
    output a slice.  The same rows copied together give bit-identical results."""
    rows, wide, hq, hkv, d = 140000, 32768, 2, 1, 64
    assert (rows - 1) * wide > 2 ** 32
    n, k0 = 300, rows - 1000
    seqs = [(0, 40, 0, 40), (rows - n, n, k0, 1000)]
    g = torch.Generator(device="cuda").manual_seed(9)
    buf = torch.empty(rows, wide, dtype=torch.bfloat16, device="cuda")   # 9.2 GB, only the sequences' rows are filled
    at = 0

    def part(heads):
        nonlocal at
        x = buf[:, at:at + heads * d].unflatten(1, (heads, d))
        at += heads * d
        return x

    Q, K, V, dO, O, dQ, dK, dV = (part(h) for h in (hq, hkv, hkv, hq, hq, hq, hkv, hkv))
    for x in (Q, K, V, dO):
        for a, b in ((0, 40), (k0, rows)):
            x[a:b] = torch.randn(x[a:b].shape, device="cuda", generator=g).bfloat16()
    _, lse = api.attn_fwd(Q, K, V, seqs, O=O)
    api.attn_bwd(dO, Q, K, V, O, lse, seqs, dQ=dQ, dK=dK, dV=dV)
    q, do = (torch.cat([x[:40], x[rows - n:]]) for x in (Q, dO))
    k, v = (torch.cat([x[:40], x[k0:]]) for x in (K, V))
    near = [(0, 40, 0, 40), (40, n, 40, 1000)]
    want = run(q, k, v, do, near, None)
    for got, ref, m in ((O, want[0], n), (dQ, want[2], n), (dK, want[3], 1000), (dV, want[4], 1000), (lse, want[1], n)):
        assert torch.equal(got[:40], ref[:40]) and torch.equal(got[rows - m:], ref[40:])
    assert not O[40:rows - n].count_nonzero() and not dK[40:k0].count_nonzero()


@pytest.mark.parametrize("lengths,hq,hkv,d,layout", [
    ([900], 8, 1, 128, "rows"), ([1500], 1, 1, 64, "heads"), ([700, 3, 0, 130, 257], 12, 1, 72, "rows"),
    ([1300, 40], 7, 1, 128, "fused"), ([513, 512, 511], 16, 2, 40, "rows"), ([260], 128, 1, 64, "rows")])
def test_few_key_heads(lengths, hq, hkv, d, layout):
    """Queries of dK and dV split over several SMs and joined: many query heads on few key heads, ends that do not fill a
    tile, unused rows between; against the formula, and against the unsplit way (a workspace without the region)."""
    seqs, rows = packed(lengths, 128)
    seqs.append((rows, 300, rows, 41))           # more queries than keys
    seqs.append((rows + 301, 5, rows + 43, 700))   # fewer
    tq, tk = rows + 310, rows + 750
    if layout == "fused":
        tq = tk = max(tq, tk)
    Q, K, V, dO = inputs(tq, tk, hq, hkv, d, layout, seed=hq)
    got = run(Q, K, V, dO, seqs, None)
    check(Q, K, V, seqs, d ** -0.5, dO, got)
    ws = torch.zeros(256 + -(-tq * hq * 4 // 256) * 256, dtype=torch.uint8, device="cuda")
    whole = api.attn_bwd(dO, Q, K, V, got[0], got[1], seqs, ws=ws)
    assert torch.equal(whole[0], got[2])
    for a, b in zip(whole[1:], got[3:]):
        assert off(a, b.double().cpu()) <= TOL
    again = api.attn_bwd(dO, Q, K, V, got[0], got[1], seqs)
    assert all(torch.equal(a, b) for a, b in zip(again, got[2:]))


@pytest.mark.parametrize("lengths,hq,hkv,d,layout", [
    ([2500], 1, 1, 128, "rows"), ([1900], 4, 1, 64, "heads"), ([1700, 3, 0, 130], 2, 2, 72, "rows"),
    ([1300, 40], 6, 1, 96, "fused"), ([3001], 16, 1, 40, "rows")])
def test_long_rows_on_few_heads(lengths, hq, hkv, d, layout):
    """Keys of whole prompts split over several SMs: some of their tiles in several pieces, some in one."""
    seqs, rows = packed(lengths, 128)
    seqs.append((rows, 300, rows, 41))             # more queries than keys
    seqs.append((rows + 301, 70, rows + 43, 1800))   # fewer
    tq, tk = rows + 375, rows + 1850
    if layout == "fused":
        tq = tk = max(tq, tk)
    Q, K, V, dO = inputs(tq, tk, hq, hkv, d, layout, seed=hq)
    got = run(Q, K, V, dO, seqs, None)
    check(Q, K, V, seqs, d ** -0.5, dO, got)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    O, lse = api.attn_fwd(Q, K, V, seqs, ws=small)
    assert off(O, got[0].double().cpu()) <= TOL and torch.equal(torch.isinf(lse), torch.isinf(got[1]))
    again = api.attn_fwd(Q, K, V, seqs)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("rows,seqs,fills", [
    (8192, [(0, 1, 0, 1)], 1), (5000, [(4999, 1, 4999, 1)], 1), (3000, [(1000, 300, 1000, 300)], 1),
    (310, [(0, 300, 0, 300)], 0), (700, [(0, 1, 0, 1), (600, 1, 600, 1), (650, 50, 650, 50)], 1),
    (600, [(0, 250, 0, 250), (256, 300, 256, 300)], 0)])
def test_unused_rows_beside_few_tokens(rows, seqs, fills):
    """Many unused rows are written by a kernel over all SMs, not by the few items of the sequences; a few cost no launch."""
    Q, K, V, dO = inputs(rows, rows, 8, 2, 64, seed=rows)
    O, dQ = torch.full_like(Q, 7), torch.full_like(Q, 7)
    dK, dV = torch.full_like(K, 7), torch.full_like(V, 7)
    lse = torch.full((rows, 8), 7.0, device="cuda")
    native.timing_begin()
    api.attn_fwd(Q, K, V, seqs, O=O, lse=lse)
    torch.cuda.synchronize()
    assert native.timing_end().get("attn_fill", (0, 0))[1] == fills
    native.timing_begin()
    api.attn_bwd(dO, Q, K, V, O, lse, seqs, dQ=dQ, dK=dK, dV=dV)
    torch.cuda.synchronize()
    assert native.timing_end().get("attn_fill", (0, 0))[1] == 2 * fills
    check(Q, K, V, seqs, 0.125, dO, (O, lse, dQ, dK, dV))


def test_no_sequence_in_a_large_buffer():
    """Heads of 8 to 1024: a block of the kernel for unused rows has several rows at a time, or several rounds a row."""
    for rows, hq, hkv, d in ((5000, 1, 1, 8), (700, 3, 1, 24), (40, 1024, 8, 16), (130, 40, 40, 128)):
        Q, K, V, dO = inputs(rows, rows, hq, hkv, d)
        O, dQ = torch.full_like(Q, 7), torch.full_like(Q, 7)
        dK, dV = torch.full_like(K, 7), torch.full_like(V, 7)
        lse = torch.full((rows, hq), 7.0, device="cuda")
        api.attn_fwd(Q, K, V, [], O=O, lse=lse)
        api.attn_bwd(dO, Q, K, V, O, lse, [], dQ=dQ, dK=dK, dV=dV)
        assert bool((lse == -math.inf).all()) and not any(x.count_nonzero() for x in (O, dQ, dK, dV))


@pytest.mark.parametrize("rows,hq,hkv,d", [(77, 4, 2, 64), (500, 8, 2, 128), (1500, 4, 1, 96), (130, 2, 2, 128)])
@pytest.mark.parametrize("spread", [1.0, 5.0, 12.0])
def test_dk_where_probability_gathers(rows, hq, hkv, d, spread):
    """The delta of dK and dV is right to fp32, however far dP - delta cancels.  dK then has two roundings to bf16, of dS and of
    the output: each at most 2^-9 = 1.95e-3 of every value, so together at most 2.8e-3 in the norm where they are independent."""
    Q, K, V, dO = inputs(rows, rows, hq, hkv, d, seed=rows)
    Q = (Q.float() * spread).bfloat16()
    seqs = [(0, rows, 0, rows)]
    O, lse, dQ, dK, dV = run(Q, K, V, dO, seqs, None)
    ref = reference(Q, K, V, seqs, d ** -0.5, dO)
    assert off(dK, ref[3]) <= 2.8e-3 and off(dV, ref[4]) <= 2.8e-3
    assert off(dQ, ref[2]) <= 1e-2


def test_a_sequence_that_does_not_fit_the_slots():
    """Few queries over many keys on one key head need more slots than there are: that sequence stays whole, the next ones are
    split all the same."""
    seqs = [(0, 890, 0, 14344), (890, 1169, 14344, 1169), (2059, 981, 15513, 981)]
    Q, K, V, dO = inputs(3040, 16494, 10, 1, 64, seed=890)
    O, lse = api.attn_fwd(Q, K, V, seqs)
    native.timing_begin()
    grads = api.attn_bwd(dO, Q, K, V, O, lse, seqs)
    torch.cuda.synchronize()
    assert native.timing_end()["attn_join"][1] == 1
    check(Q, K, V, seqs, 0.125, dO, (O, lse, *grads))
