"""Broadcast views as inputs of the tree attention: the same bits as copies of
them, in the types, head counts and widths where a tensor map's own strides
would show; broadcast caches are refused."""

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


def inputs(dtype, total, Hq, Hkv, D, page=16, lengths=(70, 0, 200)):
    g = torch.Generator().manual_seed(D + total)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    B, width = len(lengths), -(-max(lengths) // page)
    P = B * width
    cut = [total * b // B for b in range(B + 1)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    return dict(q=r(total, Hq, D), k=r(total, Hkv, D), v=r(total, Hkv, D), k_cache=r(P, page, Hkv, D), v_cache=r(P, page, Hkv, D),
                table=torch.randperm(P, generator=g).int().view(B, width).to(DEV), lengths=i32(lengths), cu_nodes=i32(cut),
                n=max(b - a for a, b in zip(cut, cut[1:])))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("total,Hq,Hkv,D", [(21, 8, 4, 128), (300, 4, 2, 64), (9, 6, 3, 80)])
@pytest.mark.parametrize("odd", [False, True])
def test_broadcast_queries_keys_and_values(dtype, total, Hq, Hkv, D, odd):
    a = inputs(dtype, total, Hq, Hkv, D)
    if odd:  # drafted values that are no numbers take a path of their own
        a["v"][total // 2, 0, 3] = float("inf")
    heads = lambda t: t[:, :1].expand(-1, t.shape[1], -1)
    rows = lambda t: t[:1].expand(t.shape[0], -1, -1)
    for shown in (dict(k=heads(a["k"])), dict(v=heads(a["v"])), dict(q=heads(a["q"])), dict(q=rows(a["q"])), dict(k=rows(a["k"]), v=rows(a["v"])),
                  dict(q=heads(rows(a["q"])), k=heads(rows(a["k"])), v=heads(rows(a["v"])))):
        got = sv().tree_attention(**{**a, **shown})
        want = sv().tree_attention(**{**a, **{n: t.contiguous() for n, t in shown.items()}})
        assert not got.status.any()
        assert torch.equal(got.out.view(torch.int16), want.out.view(torch.int16)) and torch.equal(got.lse, want.lse)


def test_broadcast_caches_are_refused():
    a = inputs(torch.bfloat16, 6, 4, 2, 64)
    for name in ("k_cache", "v_cache"):
        t = a[name]
        for view in (t[:, :, :1].expand(-1, -1, 2, -1), t[:, :1].expand(-1, 16, -1, -1), t[:1].expand(t.shape[0], -1, -1, -1)):
            with pytest.raises(ValueError, match="broadcast"):
                sv().tree_attention(**{**a, name: view})
    # one key head, shown as one: any stride
    b = inputs(torch.bfloat16, 6, 4, 1, 64)
    t = b["k_cache"]
    one = t.as_strided(t.shape, (t.stride(0), t.stride(1), 0, 1))
    assert torch.equal(sv().tree_attention(**b).out, sv().tree_attention(**{**b, "k_cache": one}).out)


def test_an_out_in_the_projection_of_its_inputs():
    """Beside q, k and v in one tensor: taken; over a part of one: refused."""
    a = inputs(torch.bfloat16, 21, 8, 4, 64)
    want = sv().tree_attention(**a)
    fused = torch.full((21, 28, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    for name, lo, hi in (("q", 4, 12), ("k", 12, 16), ("v", 16, 20)):
        fused[:, lo:hi] = a[name]
        a[name] = fused[:, lo:hi]
    got = sv().tree_attention(**a, out=fused[:, 20:])
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
    assert (fused[:, :4] == 7).all() and torch.equal(fused[:, 20:], want.out)
    kept = fused.clone()
    flat = a["k_cache"].view(-1)
    for out, name in ((fused[:, 3:11], "q"), (fused[:, 15:23], "k"), (fused[:, 17:25], "v"),
                      (flat[4096:4096 + 21 * 8 * 64].view(21, 8, 64), "k_cache")):
        with pytest.raises(sv().SVError, match=f"out shares memory with {name}"):
            sv().tree_attention(**a, out=out)
    assert torch.equal(fused, kept)
