"""GPU: the operators in a row, as a decoder layer uses them: quantized q/k/v product, the cache, attention, the output
product, the scored router and the routed experts, for a prompt and then token by token, against the same steps in
64 bits on the stages' own inputs."""
import numpy as np
import pytest
import torch

import oracle
from block_quantized_matvec_amd import ft, synth
from tests import kv_ref
from tests.gpu_util import check_fp32, dev, host, need_gpu

pytestmark = pytest.mark.gpu


def test_layer():
    need_gpu()
    H, heads, heads_kv, dim, page, E, I, topk = 512, 8, 2, 64, 16, 16, 256, 4
    g = synth.rng(77)
    n_qkv = (heads + 2 * heads_kv) * dim
    Wqkv, Wo, Wr = (synth.weights("Q4_K", n, k, g) for n, k in ((n_qkv, H), (H, heads * dim), (E, H)))
    banks = [synth.expert_bank("Q5_K", E, I, H, g), synth.expert_bank("Q5_K", E, I, H, g), synth.expert_bank("Q5_K", E, H, I, g)]
    dqkv, do, dr, dbanks = dev(Wqkv), dev(Wo), dev(Wr), [dev(b) for b in banks]
    bias = 0.01 * torch.randn(E, device="cuda")
    cache = ft.KvCache.empty(8, page, heads_kv, dim, "Q8_0", "Q4_0")
    table = torch.tensor([[5, 0, 3, 7, 1, 2, 6, 4]], dtype=torch.int32, device="cuda")
    tab = table.cpu().numpy()[0]
    keys = {"k": [], "v": []}
    done = 0
    for t in (37, 1, 1, 5, 1):
        x = dev(synth.activations(t, H, g) * np.float32(0.05))
        qkv = ft.mul_mat_vec_q("Q4_K", dqkv, n_qkv, H, "Q8_1", ft.quantize_act("Q8_1", x), t)
        q, k, v = (a.unflatten(1, (-1, dim)) for a in qkv.split([heads * dim, heads_kv * dim, heads_kv * dim], 1))
        j = np.arange(done, done + t)
        ft.kv_store(cache, k, v, torch.from_numpy(tab[j // page].astype(np.int64) * page + j % page).cuda())
        done += t
        o = ft.attn_kv(cache, q, table, torch.tensor([done], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, t], dtype=torch.int32, device="cuda"))
        y1 = ft.mul_mat_vec_q("Q4_K", do, H, heads * dim, "Q8_1", ft.quantize_act("Q8_1", o.flatten(1) * 0.01), t)
        logits = ft.mul_mat_vec_q("Q4_K", dr, E, H, "Q8_1", ft.quantize_act("Q8_1", y1), t)
        ids, w = ft.moe_route_ex(logits, topk, score="sigmoid", bias=bias, n_group=4, topk_group=2, group_top=2, scale=2.0)
        y = ft.moe_q_vec("Q5_K", *dbanks, E, H, I, "Q8_K", y1, ids, w)
        # attention on its own inputs
        keys["k"].append(kv_ref.values(*kv_ref.quantize(host(k), "Q8_0")))
        keys["v"].append(kv_ref.values(*kv_ref.quantize(host(v), "Q4_0")))
        kk, vv = np.concatenate(keys["k"]), np.concatenate(keys["v"])
        ro, terms, zero, mass = kv_ref.attention(host(q).astype(np.float64), kk, vv, t, done)
        bound = kv_ref.attention_bound(ro, terms, zero, mass, vv, "f32")
        off = np.abs(host(o) - ro)
        at = np.unravel_index(np.argmax(off / bound), off.shape)
        assert off[at] <= bound[at], f"{t} of {done} tokens, {at}: {host(o)[at]} for {ro[at]}, bound {bound[at]}, terms {terms[at[:2]]}"
        rid, rw = kv_ref.route(host(logits), topk, sigmoid=True, bias=bias.cpu().numpy(), n_group=4, topk_group=2, group_top=2, scale=2.0)
        assert np.array_equal(host(ids), rid)
        assert np.allclose(host(w), rw, rtol=2.0 ** -23, atol=0)
        ref = oracle.moe_forward("Q5_K", *banks, E, H, I, "Q8_K", host(y1), rid, host(w))["y"]
        assert np.max(np.abs(host(y) - ref)) <= 1e-2 * np.max(np.abs(ref))   # end to end, a code of h may differ
