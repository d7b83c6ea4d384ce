"""A plan that refuses a sequence, fed to the operators behind it: the other sequences' results are those of the formula
in 64 bits over their own rows, and nothing of the refused one's tokens gets into a cache.

Tolerance, for u = 2^-11 (fp16), A = sum_j p_j |v_j|: one rounding of the result, u |ref|, and one of the
probabilities, u A; scores are sums of 64 products in fp32, 2^-16 (1 + max|s|) A; fp16's smallest step 2^-24."""
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARK = 77.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("why", ["pages", "table"])
def test_a_refused_sequence_leaves_the_others_alone(why):
    page, width, heads, kv, dim = 16, 12, 8, 2, 64
    gen = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(s, device=DEV, generator=gen).half()  # noqa: E731
    turns, _ = g.rotary_table(dim)
    # a first step that fits: 30, 40 and 5 tokens in 2 + 3 + 1 of 12 pages
    lens, table, free, count = i32([0, 0, 0]), i32([[-1] * width] * 3), i32(list(range(12))), i32([12])
    caches = [torch.full((12, page, kv, dim), MARK, dtype=torch.float16, device=DEV) for _ in range(2)]
    keys, values = [[], [], []], [[], [], []]

    def step(added, tokens):
        q, k, v = rnd(tokens, heads, dim), rnd(tokens, kv, dim), rnd(tokens, kv, dim)
        before = [int(n) for n in lens]
        _, cu, pos, slots = g.page_plan(lens, i32(added), table, free, count, page_size=page, max_tokens=tokens, seq_lens=lens)
        k_out = torch.empty_like(k)
        q, k_out = g.rotary(q, k, pos, turns, v=v, k_cache=caches[0], v_cache=caches[1], slots=slots, k_out=k_out)
        out = torch.full((tokens, heads, dim), MARK, dtype=torch.float16, device=DEV)
        g.chunk_attention(q, *caches, table, lens, cu, out=out)
        for b in range(3):
            if int(lens[b]) == before[b] + added[b]:
                keys[b].append(k_out[cu[b]:cu[b + 1]])
                values[b].append(v[cu[b]:cu[b + 1]])
        return q, cu.tolist(), slots, out

    def look(q, cu, out, of):
        for b in of:
            k, v = torch.cat(keys[b]).double(), torch.cat(values[b]).double()
            x, n = q[cu[b]:cu[b + 1]].double(), k.shape[0]
            m = x.shape[0]
            s = torch.einsum("thgd,nhd->hgtn", x.reshape(m, kv, -1, dim), k) * dim ** -0.5
            hidden = torch.arange(n, device=DEV) > n - m + torch.arange(m, device=DEV)[:, None]
            p = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
            ref, A = (torch.einsum("hgtn,nhd->thgd", p, y).reshape(m, heads, dim) for y in (v, v.abs()))
            tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -16 * (1 + float(s.abs().max()))) * A + 2.0 ** -24
            assert bool(((out[cu[b]:cu[b + 1]].double() - ref).abs() <= tol).all()), b

    q, cu, _, out = step([30, 40, 5], 80)
    assert g.device_status() == 0
    look(q, cu, out, range(3))
    assert bool((out[75:] == MARK).all())
    # the second asks for more than there is, between two that get what they ask for
    held = [c[table[1, :3].long()].clone() for c in caches]
    many = 152 if why == "pages" else 153             # of 40: 192 tokens in 9 pages more, where 4 are left; 193 of 192
    q, cu, slots, out = step([20, many, 2 if why == "pages" else 30], 30 + many + 30)
    assert g.device_status() == (g.DEV_NO_PAGE if why == "pages" else g.DEV_SEQ_LEN)
    assert lens.tolist() == [50, 40, 7 if why == "pages" else 35] and bool((slots[cu[1]:cu[2]] == -1).all())
    look(q, cu, out, (0, 2))
    for c, before in zip(caches, held):
        assert torch.equal(c[table[1, :3].long()], before)
    used = torch.cat([table[0, :4], table[1, :3], table[2, :1 if why == "pages" else 3]]).long()
    rest = torch.ones(12, dtype=torch.bool, device=DEV)
    rest[used] = False
    for c in caches:
        assert bool((c[rest] == MARK).all())
    assert sorted(free[:int(count)].tolist()) == rest.nonzero().flatten().tolist()
