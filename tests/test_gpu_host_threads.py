"""GPU: several host threads call on one stream (torch's threads share the default one): each call's launches stay
together on it, so none reads what another wrote to the stream's scratch pool between them."""
import threading

import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft, synth
from tests.gpu_util import dev, need_gpu
from tests.test_gpu_attn_kv import build, ints

pytestmark = pytest.mark.gpu


def together(calls, rounds=60):
    """Each call in a thread of its own, over and over; every output is the one of the call made alone."""
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors = [[] for _ in calls], []
    gate = threading.Barrier(len(calls))

    def work(i):
        try:
            gate.wait(30)
            for _ in range(rounds):
                got[i].append(calls[i]())
        except Exception as e:  # noqa: BLE001 - shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not errors and all(len(g) == rounds for g in got), errors
    for w, outs in zip(want, got):
        for o in outs:
            assert torch.equal(o, w)


def test_attention_with_split_keys():
    need_gpu()
    calls = []
    for seed in range(4):
        kv = [2000, 900 + seed]
        cache, table, _ = build(kv, 2, 64, 32, "Q8_0", "Q8_0", seed)
        q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(seed)).cuda()
        calls.append(lambda a=(cache, q, table, ints(kv), ints([0, 1, 2])): ft.attn_kv(*a, max_kv=2000))
    together(calls)


def test_repacked_activations():
    need_gpu()
    calls = []
    for seed in range(4):
        g = synth.rng(900 + seed)
        W = dev(synth.weights("Q4_0", 256, 512, g))
        xq = ft.quantize_act("Q8_0", dev(synth.activations(3, 512, g)))
        calls.append(lambda W=W, xq=xq: ft.mul_mat_vec_q("Q4_0", W, 256, 512, "Q8_0", xq, 3))
    together(calls)


def test_layers_and_grouped_products():
    need_gpu()
    calls = []
    E, H, I, K = 8, 512, 256, 2
    for seed in range(3):
        g = synth.rng(910 + seed)
        banks = [dev(synth.expert_bank("Q4_K", E, I, H, g)), dev(synth.expert_bank("Q4_K", E, I, H, g)), dev(synth.expert_bank("Q4_K", E, H, I, g))]
        x = dev(synth.activations(20, H, g) * np.float32(0.05))
        ids, w = dev(synth.expert_ids(20, E, K, g)), dev(synth.expert_weights(20, K, g))
        calls.append(lambda b=banks, x=x, ids=ids, w=w: ft.moe_q_vec("Q4_K", *b, E, H, I, "Q8_K", x, ids, w))
    together(calls)
