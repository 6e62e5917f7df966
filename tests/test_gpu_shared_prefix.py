"""The example that runs append, rotation and attention over a shared prefix together: at every step the new
queries are rotated by the formula, and the answers are plain attention over the cells that the pages hold."""
import os
import sys

import pytest
import torch

import cache_ref as ref
import token_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
def test_example_agrees_with_plain_attention(int8):
    import shared_prefix as ex
    seen = []
    texts, readers, question, nkv, group, page = 2, 5, 7, 2, 4, 16

    def each_step(s):
        torch.cuda.synchronize()
        n = question + len(seen) + 1
        assert s["lens"].tolist() == [n] * (texts * readers)
        want = [s["text_lens"][i // readers] + n - 1 for i in range(texts * readers)]
        assert s["at"].tolist() == want
        q = token_ref.rotate(s["q"], s["at"], s["freqs"])
        tol = token_ref.rotate_tol(s["q"], q, torch.bfloat16, 64)
        assert bool(((s["turned_q"].cpu().double() - q).abs() <= tol).all())
        p_half = 2.0 ** -11 if int8 else 2.0 ** -8
        for i in (0, 3, readers, texts * readers - 1):
            for h in range(nkv):
                def cells(pool, scale, row, m):
                    return ref.paged_cells(s[pool], s.get(scale), row, m, h, page)[0]
                t, m = i // readers, s["text_lens"][i // readers]
                k = torch.cat((cells("k", "k_scale_f16", s["text_table"][t], m), cells("k", "k_scale_f16", s["own_table"][i], n)))
                v = torch.cat((cells("v", "v_scale_f16", s["text_table"][t], m), cells("v", "v_scale_f16", s["own_table"][i], n)))
                every = torch.ones((1, m + n), dtype=torch.bool, device=k.device)
                hs = slice(h * group, (h + 1) * group)
                o, l, _, size, S = ref.attend(s["turned_q"][i, hs][:, None], k, v, every, 128 ** -0.5)
                bound, _ = ref.bounds(o, l, size, S, m + n, torch.bfloat16, p_half)
                if int8:    # binary16 weights below its normal numbers: see test_gpu_prefix_attn
                    bound = bound + 2 * (m + n) * 2.0 ** -32 * size.amax(-1, keepdim=True)
                ref.check(s["out"][i, hs], o[:, 0], bound[:, 0], (len(seen), i, h))
        seen.append(n)

    out = ex.generate(texts=texts, readers=readers, text=300, question=question, steps=25, heads=nkv * group, nkv=nkv, page=page, int8=int8,
                      each_step=each_step)
    assert len(seen) == 25 and torch.isfinite(out).all()


@pytest.mark.parametrize("texts,text", [(4, 150), (3, 1)])
def test_example_with_more_texts_than_hundreds_of_tokens(texts, text):
    """Further texts are shorter, down to one token, whose value its readers weigh beside their own cells."""
    import shared_prefix as ex
    last = {}

    def each_step(s):
        last.update(s)

    out = ex.generate(texts=texts, readers=2, text=text, question=3, steps=2, heads=4, nkv=1, each_step=each_step)
    assert last["text_lens"] == [max(1, text - 100 * t) for t in range(texts)] and min(last["text_lens"]) == 1
    for i in range(2 * texts):
        m, n = last["text_lens"][i // 2], 5
        assert int(last["lens"][i]) == n and int(last["at"][i]) == m + n - 1
        k, v = (torch.cat((ref.paged_cells(last[x], None, last["text_table"][i // 2], m, 0, 16)[0],
                           ref.paged_cells(last[x], None, last["own_table"][i], n, 0, 16)[0])) for x in ("k", "v"))
        o, l, _, size, S = ref.attend(last["turned_q"][i][:, None], k, v, torch.ones((1, m + n), dtype=torch.bool, device=k.device), 128 ** -0.5)
        bound, _ = ref.bounds(o, l, size, S, m + n, torch.bfloat16, 2.0 ** -8)
        ref.check(out[i], o[:, 0], bound[:, 0], i)
