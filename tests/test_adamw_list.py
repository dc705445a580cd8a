"""The tensors of an AdamW list are checked against its counts: a count beyond
a tensor's end would have the step read and write whatever lies behind it."""
import pytest
import torch

import long_context_lm_rel_gb300 as rxl


def entry(n, bits=32, device="cpu", **kw):
    state = dict(dtype=torch.uint8) if bits == 8 else {}
    z = lambda k, **a: torch.zeros(k, device=device, **a)  # noqa: E731
    t = dict(param=z(n, dtype=torch.bfloat16), grad=z(n, dtype=torch.bfloat16), master=z(n), m=z(n, **state),
             v=z(n, **state), n=n)
    if bits == 8:
        t.update(m_scale=z(-(-n // 128)), v_scale=z(-(-n // 128)))
    return {**t, **kw}


@pytest.mark.parametrize("name", ["param", "master", "grad", "m", "v"])
@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_that_are_too_short(name, bits):
    t = entry(300, bits)
    t[name] = t[name][:299]
    with pytest.raises(ValueError, match=f"{name} has 299 elements where 300"):
        rxl.make_adamw_tensors(rxl.make_adamw_desc(state_bits=bits), [t])


@pytest.mark.parametrize("name", ["m_scale", "v_scale"])
def test_scales_of_a_ragged_count(name):
    t = entry(300, 8, **{name: torch.zeros(300 // 128)})
    with pytest.raises(ValueError, match=f"{name} has 2 elements where 3"):
        rxl.make_adamw_tensors(rxl.make_adamw_desc(state_bits=8), [t])


@pytest.mark.parametrize("name", ["param", "master", "grad", "m", "v", "m_scale", "v_scale"])
def test_tensors_with_gaps(name):
    t = entry(256, 8)
    wide = torch.zeros(2 * t[name].numel(), dtype=t[name].dtype)
    t[name] = wide[::2]
    with pytest.raises(ValueError, match=f"{name} is not contiguous"):
        rxl.make_adamw_tensors(rxl.make_adamw_desc(state_bits=8), [t])


def test_tensors_in_different_orders():
    t = entry(12)
    t["param"] = torch.zeros(4, 3, dtype=torch.bfloat16).t()
    with pytest.raises(ValueError, match="param is not contiguous"):
        rxl.make_adamw_tensors(rxl.make_adamw_desc(), [t])
    t = {k: x.view(4, 3).t() if k != "n" else x for k, x in entry(12).items()}
    t["grad"] = t["grad"].contiguous()
    with pytest.raises(ValueError, match="not contiguous"):
        rxl.make_adamw_tensors(rxl.make_adamw_desc(), [t])
    gaps = {k: torch.zeros(3, 8, dtype=x.dtype).t()[:4] if k != "n" else x for k, x in entry(12).items()}
    with pytest.raises(ValueError, match="not contiguous"):
        rxl.make_adamw_tensors(rxl.make_adamw_desc(), [gaps])


def test_addresses_and_empty_entries_pass():
    rxl.build()
    a = 1 << 20
    out = rxl.make_adamw_tensors(rxl.make_adamw_desc(), [dict(param=a, grad=a + 64, m=a + 128, v=a + 192, n=5),
                                                         dict(param=a, grad=a, m=a, v=a, n=0)])
    assert (out[0].param, out[0].grad, out[0].m, out[0].v, out[0].n, out[1].n) == (a, a + 64, a + 128, a + 192, 5, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_lists_that_fit(bits):
    """Longer tensors than the count, flat states of a matrix, and matrices that all lie transposed."""
    desc, n = rxl.make_adamw_desc(state_bits=bits), 21 * 37
    rand = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).bfloat16()
    plain = entry(n, bits, "cuda", grad=rand)
    matrix = {**entry(n, bits, "cuda"), "grad": rand.clone().view(21, 37)}
    matrix["param"] = matrix["param"].view(21, 37)
    turned = {k: x.view(37, 21).t() if k in ("param", "master", "grad", "m", "v") else x
              for k, x in entry(n, bits, "cuda", grad=rand.clone()).items()}
    longer = {**entry(n + 200, bits, "cuda"), "n": n}
    longer["grad"][:n] = rand
    longer["grad"][n:] = 1
    for t in (plain, matrix, turned, longer):  # each alone: the rounding by chance depends on the place in the list
        rxl.rxl_adamw_step(desc, rxl.make_adamw_tensors(desc, [t]), 1, rxl.rxl_adamw_scalars_at(desc, 1, 1e-2), None)
    for k in ("param", "master", "m", "v"):
        want = plain[k]
        assert want.any()
        assert torch.equal(matrix[k].reshape(-1), want) and torch.equal(turned[k].t().reshape(-1), want)
        assert torch.equal(longer[k][:n], want) and not longer[k][n:].any(), k
