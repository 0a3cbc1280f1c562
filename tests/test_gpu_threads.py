"""Attention and losses called from several host threads without a workspace of the caller's."""
import threading

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api  # noqa: E402


def loss_inputs(rows, vocab, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn(rows, vocab, device="cuda", generator=g) * 3).to(dtype)
    y = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    return z, y, torch.randn(3, rows, device="cuda", generator=g)


def preference(rows, vocab, dtype, n_pairs, seed):
    z, y, noise = loss_inputs(rows, vocab, dtype, seed)
    each = rows // (2 * n_pairs)
    pairs = api.pref_pairs([(2 * i * each, (2 * i + 1) * each, each, each) for i in range(n_pairs)])
    return lambda: api.pref_loss(z, y, pairs, noise[0].contiguous(), beta=0.3, label_smoothing=0.1)


def policy(rows, vocab, dtype, seed):
    z, y, noise = loss_inputs(rows, vocab, dtype, seed)
    return lambda: api.policy_loss(z, y, noise[0] - 8, noise[1], noise[2] - 8, kl_coef=0.1)


def attention(seqs, hq, hkv, d, seed):
    """Forward and backward; the sequences' keys (and queries) are split over several SMs."""
    rows, k_rows = max(s[0] + s[1] for s in seqs), max(s[2] + s[3] for s in seqs)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, d_o = (torch.randn(rows, hq, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    k, v = (torch.randn(k_rows, hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    table = api.attn_seqs(seqs)

    def call():
        o, lse = api.attn_fwd(q, k, v, table)
        return (o, lse, *api.attn_bwd(d_o, q, k, v, o, lse, table))

    return call


def test_threads_on_one_stream():
    """Each thread's results are those of the same calls made alone."""
    makers = [lambda: attention([(0, 1, 0, 6000)], 8, 2, 64, 1), lambda: attention([(0, 1500, 0, 1500)], 8, 1, 64, 2),
              lambda: preference(300, 5000, torch.bfloat16, 70, 3), lambda: policy(60, 32001, torch.bfloat16, 4)]
    work = [m() for m in makers]
    want = [[x.clone() for x in f()] for f in work]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(work))

    def run(i):
        try:
            start.wait(60)
            for _ in range(40):
                if not all(torch.equal(a, b) for a, b in zip(want[i], work[i]())):
                    wrong.append(i)
        except Exception as e:   # reported by the main thread
            wrong.append((i, e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
