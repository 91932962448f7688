"""The example's attention block (W12 products around the paged cache) over a few
steps with drafted tokens, against a plain torch layer on the same BF16 weights that
keeps the accepted tokens' keys and values in lists."""
import importlib.util
import os

import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVPages, w12

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from gpu_util import ensure_built
    ensure_built()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(x, w):
    x = x.double()
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()


def rotate(x, rope, pos):
    half = rope.shape[1] // 2
    c, s = rope[pos, :half].double()[:, None], rope[pos, half:].double()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def bf(x):
    return x.to(torch.bfloat16).double()


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("heads,kv_heads,dim,per", [(6, 2, 64, 3), (12, 1, 128, 5)])
def test_block_against_plain_layer(example, cache, heads, kv_heads, dim, per):
    hidden, requests, steps = 256, 3, 9
    pages = KVPages.create(64, 16, requests, 16)
    block, (wq, wk, wv, wo), (qn, kn) = example.make_block(hidden, heads, kv_heads, dim, pages, 64, cache)
    rope = example.rope_table(256, dim)
    step = pages.step(requests * per, max_new=per)
    lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
    new = torch.full_like(lens, per)
    g = torch.Generator(device="cuda").manual_seed(2)
    kept = [(torch.zeros(0, kv_heads, dim, device="cuda", dtype=torch.float64),) * 2 for _ in range(requests)]
    for _ in range(steps):
        x = torch.randn(requests * per, hidden, device="cuda", generator=g).to(torch.bfloat16)
        pages.plan(lens, new, step)
        y = block(x, step, rope)
        w12.w12_check_status()
        accepted = torch.randint(1, per + 1, (requests,), device="cuda", generator=g, dtype=torch.int32)
        xd = x.double()
        want = []
        for b in range(requests):
            rows = xd[b * per:(b + 1) * per]
            pos = torch.arange(per, device="cuda") + int(lens[b])
            q = bf(rotate(norm(bf(rows @ wq.double().T).view(per, heads, dim), qn), rope, pos))
            k = rotate(norm(bf(rows @ wk.double().T).view(per, kv_heads, dim), kn), rope, pos)
            v = bf(rows @ wv.double().T).view(per, kv_heads, dim)
            ks, vs = torch.cat([kept[b][0], bf(k)]), torch.cat([kept[b][1], v])
            out = []
            for i in range(per):
                n = kept[b][0].shape[0] + i + 1
                s = torch.einsum("hgd,khd->hgk", q[i].view(kv_heads, -1, dim), ks[:n]) * dim ** -0.5
                out.append(torch.einsum("hgk,khd->hgd", torch.softmax(s, -1), vs[:n]).reshape(-1))
            want.append(rows + bf(torch.stack(out)) @ wo.double().T)
            a = int(accepted[b])
            kept[b] = (ks[:len(ks) - per + a], vs[:len(vs) - per + a])
        want = torch.cat(want)
        # BF16 steps (q/k/v, softmax weights, output, product) of 2^-8 each, about 2^-9
        # rms; an 8-bit cache adds a step of 1/254 of each row's largest value
        err = float((y.double() - want).norm() / want.norm())
        assert err < (0.01 if cache == "bf16" else 0.02), err
        lens += accepted
    assert pages.owned.tolist() == [-(-(n + per - int(a)) // 16) for n, a in zip(lens.tolist(), accepted.tolist())]


def test_example_runs(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["decode_layer.py", "--steps", "5", "--cache", "q8"])
    example.main()
    assert "pages free again" in capsys.readouterr().out
