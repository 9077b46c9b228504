"""The 64-bit attention over packed sequences that the GPU tests compare with: against the dense oracle sequence by
sequence, and its gradients against differences."""

import numpy as np
import pytest

import oracle
import packed_util as pu


class HostBatch:
    """packed_util.Batch without a device."""

    def __init__(self, lens, Hq, Hkv, d, seed, lead=0, tail=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.cu = lens, Hq, Hkv, d, pu.starts(lens, lead)
        self.rows = int(self.cu[-1]) + tail
        self.q, self.do = (rng.standard_normal((self.rows, Hq, d)) for _ in range(2))
        self.k, self.v = (rng.standard_normal((self.rows, Hkv, d)) for _ in range(2))

    sequences, held = pu.Batch.sequences, pu.Batch.held


@pytest.mark.parametrize("causal", [False, True])
def test_sequences_are_the_dense_oracles(causal):
    b = HostBatch([5, 0, 1, 9], 4, 2, 8, 1, lead=2, tail=3)
    o, lse, _, _ = pu.forward_ref(b, causal, 0.3)
    grads, _ = pu.backward_ref(b, o, lse, causal, 0.3)
    assert np.isnan(o[~b.held()]).all() and not np.isnan(o[b.held()]).any()
    for r in b.sequences():
        q, k, v, do = (t[r].swapaxes(0, 1)[None] for t in (b.q, b.k, b.v, b.do))
        o_ref, l_ref = oracle.attention_forward(q, k, v, causal, 0.3)
        assert np.allclose(o[r].swapaxes(0, 1), o_ref[0], atol=1e-12)
        assert np.allclose(lse[:, r], l_ref[0], atol=1e-12)
        for g, ref in zip(grads, oracle.attention_backward(q, k, v, do, causal, 0.3)):
            assert np.allclose(g[r].swapaxes(0, 1), ref[0], atol=1e-11)


@pytest.mark.parametrize("causal", [False, True])
def test_gradients_match_differences(causal):
    b = HostBatch([4, 1, 6], 2, 1, 5, 2)

    def loss():
        return float((pu.forward_ref(b, causal, 0.4)[0] * b.do).sum())

    o, lse, _, _ = pu.forward_ref(b, causal, 0.4)
    grads, _ = pu.backward_ref(b, o, lse, causal, 0.4)
    rng, h = np.random.default_rng(3), 1e-5
    for t, g in zip((b.q, b.k, b.v), grads):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in t.shape)
            was = t[at]
            t[at] = was + h
            up = loss()
            t[at] = was - h
            down = loss()
            t[at] = was
            assert abs((up - down) / (2 * h) - g[at]) <= 1e-7 * max(1.0, abs(g[at]))
