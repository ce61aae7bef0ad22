"""GPU checks of the norm's cached form in batches of more requests than its
kernel keeps the offsets of, and of calls at the same time."""

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa

from test_qk_norm import EPS, Case, cache_of, dev, freqs, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,total", [(1023, 1000), (1024, 1000), (5000, 4000), (3000, 20000)])
def test_append_of_many_requests_equals_the_two_calls(cuda_device, B, total):
    """Requests without tokens among them; positions beyond 2^24."""
    rng = np.random.default_rng(B)
    d, bs, Hq, Hkv = 64, 16, 3, 2
    cu = np.concatenate([[0], np.sort(rng.integers(0, total + 1, B - 1)), [total]])
    used = -(-np.diff(cu) // bs)
    start = np.concatenate([[0], np.cumsum(used)])
    perm = rng.permutation(int(used.sum()) + 1)
    slots = np.concatenate([perm[start[b] + np.arange(n) // bs] * bs + np.arange(n) % bs
                            for b, n in enumerate(np.diff(cu))])
    q, k, v = dev(rng.normal(size=(total, Hq + 2 * Hkv, d)), cuda_device, torch.bfloat16).split([Hq, Hkv, Hkv], 1)
    w = dev(1 + 0.2 * rng.normal(size=d), cuda_device, torch.bfloat16)
    kw = dict(inv_freq=dev(freqs(d), cuda_device, torch.float64), eps=EPS, q_weight=w, k_weight=w,
              cu_seqlens=dev(cu, cuda_device, torch.int32),
              ends=dev(rng.integers(0, 1 << 30, B), cuda_device, torch.int32))
    ids = dev(slots, cuda_device, torch.int32)
    ours = cache_of(rng, len(perm), Hkv, bs, d, cuda_device)
    theirs = [x.clone() for x in ours]
    q_out = fa.qk_norm_rope_append(q, k, v, *ours, ids, **kw)
    qn, kn = fa.qk_norm_rope(q, k, **kw)
    fa.cache_append(kn, v.contiguous(), *theirs, ids)
    assert torch.equal(q_out, qn)
    same(ours, theirs)


def test_gradients_at_the_same_time(cuda_device):
    """On streams of their own, each with its workspace: the bits of a call alone."""
    cases = [Case(cuda_device, "packed", d, d, Hq, Hkv, False, "qk", dtype, lens=(n, 7, n))
             for d, Hq, Hkv, dtype, n in ((128, 32, 8, torch.bfloat16, 500), (64, 9, 3, torch.float32, 90),
                                          (128, 4, 4, torch.bfloat16, 1500))]
    ins = [(c.split(c.qkv), c.split(c.up)) for c in cases]

    def call(c, x, up, **more):
        return fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw, **more)

    want = [call(c, x, up) for c, (x, up) in zip(cases, ins)]
    got = [[torch.empty_like(t) for t in w] for w in want]
    spaces = [fa.workspace(fa.qk_norm_rope_bwd_workspace_size(c.d), cuda_device) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, (x, up), g, ws, s in zip(cases, ins, got, spaces, streams):
            call(c, x, up, dq=g[0], dk=g[1], dq_weight=g[2], dk_weight=g[3], ws=ws, stream=s)
    torch.cuda.synchronize()
    for c, w, g in zip(cases, want, got):
        there = torch.tensor(c.there, device=cuda_device)
        assert torch.equal(w[0][there], g[0][there]) and torch.equal(w[1][there], g[1][there])
        assert torch.equal(w[2], g[2]) and torch.equal(w[3], g[3])
