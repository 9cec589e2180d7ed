"""The scratch size of ft.attn_kv grows with the bound of the lengths (host arithmetic, no GPU)."""
import ctypes
import random

import pytest

from block_quantized_matvec_amd import ft


def size(n_tok, n_head, n_seq, max_kv, heads_kv=8, dim=128, page=16, window=0, prefix=False, shared=0, causal=True):
    c = ft._KvCache(1, 1, 1 << 20, 1 << 20, 1 << 20, page, heads_kv, dim)
    o = ft._AttnOpts(0.0, 0.0, not causal, window, None, 1 << 20 if prefix else None, shared, None, 0)
    return ft.lib().ft_attn_kv_scratch_bytes(ctypes.byref(c), n_tok, n_head, n_seq, max_kv, ctypes.byref(o))


@pytest.mark.parametrize("seed", range(8))
def test_grows_with_the_bound(seed):
    """With few rows per sequence; with many the call takes as many parts as it has room for."""
    r = random.Random(seed)
    for _ in range(300):
        heads_kv, group, n_seq = r.choice([1, 2, 4, 8]), r.choice([1, 2, 4, 8]), r.choice([1, 1, 2, 3, 8, 32])
        n_tok = n_seq * r.randint(1, max(1, 32 // group))
        shared = r.choice([0, 0, 16 * r.randint(1, 600)])
        window = r.choice([0, 0, r.randint(1, 5000)])
        kw = dict(heads_kv=heads_kv, dim=r.choice([64, 96, 128, 256]), window=window, prefix=r.random() < 0.3, shared=shared, causal=r.random() < 0.8)
        bounds = sorted(shared + r.randint(0, r.choice([300, 3000, 140000])) for _ in range(6))
        sizes = [size(n_tok, heads_kv * group, n_seq, n, **kw) for n in bounds]
        assert sizes == sorted(sizes), (n_tok, group, n_seq, bounds, kw)
