"""GPU: a decoder layer's operators in a row, as a user's program calls them: norm and quantizer, the q/k/v product with
adapters beside it, queries and keys turned and stored, attention over the cache, the output product with adapters, the
norm after it with a gate and the residual, norm and quantizer for the next product; for prompts of two requests, then
tokens of both.  Each stage is held against its definition on its own inputs."""
import numpy as np
import pytest
import torch

import oracle
from block_quantized_matvec_amd import ft, synth
from tests import kv_ref, layer_ref as ref
from tests.gpu_util import dev, host, need_gpu
from tests.test_gpu_lora import check as check_lora

pytestmark = pytest.mark.gpu


def test_layer():
    need_gpu()
    H, heads, heads_kv, dim, page, rot, rank, many = 512, 8, 2, 64, 16, 32, 8, 3
    g = synth.rng(91)
    rs = np.random.RandomState(92)
    n_qkv = (heads + 2 * heads_kv) * dim
    Wqkv, Wo = (synth.weights("Q4_K", n, k, g) for n, k in ((n_qkv, H), (H, heads * dim)))
    dqkv, do = dev(Wqkv), dev(Wo)
    vec = lambda n, m=1.0: (m + 0.2 * rs.randn(n)).astype(np.float32)  # noqa: E731
    w_in, w_post, w_next, qw, kw = vec(H), vec(H), vec(H), vec(dim), vec(dim)
    gate = dev(vec(H, 0.5))
    mats = {}
    for name, n, k in (("qkv", n_qkv, H), ("o", H, heads * dim)):
        mats[name] = [dev((rs.randn(many, rank, k) * 0.05).astype(np.float32)).bfloat16(), dev((rs.randn(many, n, rank) * 0.05).astype(np.float32)).bfloat16()]
    scales = dev(np.array([1.0, 0.5, 2.0], np.float32))
    freqs, m = ft.rope_freqs(rot, 10000.0, "ramp", 4.0, 64)
    tab = ft.rope_table(256, freqs, m)
    cache = ft.KvCache.empty(12, page, heads_kv, dim, "Q8_0", "Q4_0")
    table = torch.tensor([[5, 0, 3, 7, 1], [2, 6, 4, 11, 8]], dtype=torch.int32, device="cuda")
    tb = host(table).astype(np.int64)
    done, keys = [0, 0], [[[], []], [[], []]]
    request = np.array([2, -1], np.int32)   # the first request's adapter; the second has none
    for new in ([37, 20], [1, 1], [1, 1], [3, 1]):
        t = sum(new)
        x = dev(synth.activations(t, H, g) * np.float32(0.05))
        seq = np.repeat([0, 1], new)
        pos = np.concatenate([np.arange(d, d + n) for d, n in zip(done, new)]).astype(np.int32)
        slots = tb[seq, pos // page] * page + pos % page
        ids = dev(request[seq])
        _, xn, xq = ft.norm(x, weight=dev(w_in), act="Q8_1", rows=True)
        base = ft.mul_mat_vec_q("Q4_K", dqkv, n_qkv, H, "Q8_1", xq, t)
        qkv = ft.lora(xn, *mats["qkv"], ids, y=base, scales=scales)
        q, k, v = (a.unflatten(1, (-1, dim)) for a in qkv.split([heads * dim, heads_kv * dim, heads_kv * dim], 1))
        qr = ft.kv_store_rope(cache, q, k, v, dev(slots), dev(pos), tab, q_weight=dev(qw), k_weight=dev(kw))
        done = [d + n for d, n in zip(done, new)]
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        o = ft.attn_kv(cache, qr, table, dev(np.array(done, np.int32)), dev(start))
        oq = ft.quantize_act("Q8_1", o.flatten(1))
        ob = ft.mul_mat_vec_q("Q4_K", do, H, heads * dim, "Q8_1", oq, t)
        out = ft.lora(o.flatten(1), *mats["o"], ids, y=ob, scales=scales, out=ob.clone())
        r, n, rq = ft.norm(out, weight=dev(w_next), residual=x, post_weight=dev(w_post), gate=gate, scale=0.5, act="Q8_K", rows=True)

        one = ref.norm(host(x), eps=1e-6, weight=w_in, at=np.float32)
        assert np.array_equal(host(xn), one) and np.array_equal(host(xq), oracle.quantize("Q8_1", one))
        f = lambda a: a.double().cpu().numpy()  # noqa: E731
        check_lora(qkv, xn, *mats["qkv"], ids, base, scales)
        turned = [ref.turn(host(a), pos, host(tab), False, w, 1e-6, np.float32) for a, w in ((q, qw), (k, kw))]
        assert np.array_equal(host(qr), turned[0])
        for i in range(2):
            mine = seq == i
            keys[i][0].append(kv_ref.values(*kv_ref.quantize(turned[1][mine], "Q8_0")))
            keys[i][1].append(kv_ref.values(*kv_ref.quantize(host(v)[mine], "Q4_0")))
            kk, vv = (np.concatenate(a) for a in keys[i])
            ro, terms, zero, mass = kv_ref.attention(f(qr)[mine], kk, vv, new[i], done[i])
            assert np.all(np.abs(f(o)[mine] - ro) <= kv_ref.attention_bound(ro, terms, zero, mass, vv, "f32"))
        check_lora(out, o.flatten(1), *mats["o"], ids, ob, scales)
        r1, n1 = ref.block(host(out), residual=host(x), post=True, post_weight=w_post, gate=host(gate), scale=0.5, eps=1e-6, weight=w_next, at=np.float32)
        assert np.array_equal(host(r), r1) and np.array_equal(host(n), n1) and np.array_equal(host(rq), oracle.quantize("Q8_K", n1))
