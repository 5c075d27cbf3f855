"""GPU parity of the gradient norm and the clipping against float64.

Tolerances: squares and sums are fp64, so the norm is off by its rounding to
fp32, 2^-24; a clipped value by its type's rounding (2^-24 fp32, 2^-8 bf16)
and, in bf16, by two roundings of the fp32 product and its factor, 2^-23."""
import numpy as np
import pytest

from oracle import step_ops as so
from tests.gpu_util import down, note, torch_dev

pytestmark = pytest.mark.gpu
ROOM = {"f32": 2.0 ** -24 * (1 + 1e-6), "bf16": 2.0 ** -8 * (1 + 1e-6) + 2.0 ** -23}


def _msr():
    import retnet_scale_retention_amd as msr
    return msr


def make(torch, dev, sizes, seed=0, size=1e-2):
    gen = torch.Generator(device=dev).manual_seed(seed)
    kinds = {"f32": torch.float32, "bf16": torch.bfloat16}
    return [(size * torch.randn(n, generator=gen, device=dev)).to(kinds[t]) for n, t in sizes], [t for _, t in sizes]


def check(torch, got, norm, grads, kinds, limit, given=False):
    want, n = so.clip([down(g) for g in grads], limit)
    assert abs(float(norm) - n) <= 2.0 ** -24 * (1 + 1e-6) * n
    # a norm that is given was rounded to fp32 before it divides: |n' / n - 1| <= 2^-24, and so is the factor's error
    more = 2.0 ** -24 * (1 + 1e-6) if given else 0.0
    for a, b, t, g in zip(got, want, kinds, grads):
        assert a.dtype == g.dtype and a.shape == g.shape
        assert np.all(np.abs(down(a) - b) <= (ROOM[t] + more) * np.abs(b) + 1e-38)


LISTS = {
    "one": [(1, "f32")],
    "empty among": [(0, "bf16"), (5, "bf16"), (0, "f32")],
    "chunk's ends": [(8191, "f32"), (8192, "f32"), (8193, "bf16"), (8192, "bf16"), (16384, "bf16"), (24577, "f32")],
    "many": [(1 + 37 * i % 9000, "bf16" if i % 3 else "f32") for i in range(400)],
    "large": [(9_000_001, "f32"), (20_000_000, "bf16"), (7, "f32")],
}


@pytest.mark.parametrize("name", sorted(LISTS))
def test_norm_and_clip(name):
    torch, dev = torch_dev()
    msr = _msr()
    note("clip", name)
    grads, kinds = make(torch, dev, LISTS[name])
    norm = msr.msr_gradient_norm(grads)
    n = float(norm)
    assert norm.shape == () and norm.dtype == torch.float32
    for limit in (0.3 * n, 2 * n, 0.0, float("inf")):
        keep = [g.clone() for g in grads]
        out, got = msr.msr_clip_gradients(grads, limit, out=[torch.full_like(g, 7) for g in grads])
        assert float(got) == n and all(torch.equal(a, b) for a, b in zip(grads, keep))
        check(torch, out, got, grads, kinds, np.float32(limit))
        # in place; with the norm given
        r, got = msr.msr_clip_gradients(keep, limit)
        assert r[0] is keep[0] and float(got) == n and all(torch.equal(a, b) for a, b in zip(keep, out))
        keep = [g.clone() for g in grads]
        _, same = msr.msr_clip_gradients(keep, limit, norm=norm)
        assert same is norm
        check(torch, keep, norm, grads, kinds, np.float32(limit), given=True)
    joined = norm * 3  # as over processes
    keep = [g.clone() for g in grads]
    msr.msr_clip_gradients(keep, n, norm=joined)
    for a, g, t in zip(keep, grads, kinds):
        f = float(np.float32(n)) / float(joined)
        assert np.all(np.abs(down(a) - down(g) * f) <= ROOM[t] * np.abs(down(g) * f) + 1e-38)


def test_views_of_one_buffer_and_shapes():
    torch, dev = torch_dev()
    msr = _msr()
    for dtype, kind in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        flat = torch.randn(100003, device=dev).to(dtype)
        cuts = [0, 1, 4, 9, 8300, 30001, 99999]
        grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
        ref = [g.clone() for g in grads]
        _, norm = msr.msr_clip_gradients(grads, 1.5)
        check(torch, grads, norm, ref, [kind] * len(grads), 1.5)
        assert bool((flat[99999:] != 0).any())
    m = [torch.randn(3, 5, 7, device=dev), torch.randn((), device=dev)]
    out, norm = msr.msr_clip_gradients(m, 0.5, out=[torch.empty_like(t) for t in m])
    assert out[0].shape == (3, 5, 7) and out[1].shape == ()
    check(torch, out, norm, m, ["f32", "f32"], 0.5)


def test_large_small_and_non_finite_gradients():
    torch, dev = torch_dev()
    msr = _msr()
    big = [torch.full((9000,), 3e36, device=dev), torch.full((77,), -1e30, device=dev, dtype=torch.bfloat16)]
    out, norm = msr.msr_clip_gradients([g.clone() for g in big], 1.0)
    check(torch, out, norm, big, ["f32", "bf16"], 1.0)
    tiny = [torch.full((9000,), 1e-30, device=dev)]
    assert abs(float(msr.msr_gradient_norm(tiny)) / (1e-30 * 9000 ** 0.5) - 1) < 1e-6
    zero = [torch.zeros(10, device=dev)]
    out, norm = msr.msr_clip_gradients(zero, 1.0)
    assert float(norm) == 0 and not out[0].any()
    for bad in (float("nan"), float("inf")):
        g = [torch.randn(20000, device=dev), torch.randn(5, device=dev).bfloat16()]
        g[0][12345] = bad
        ref = [t.clone() for t in g]
        same = lambda a, b: torch.equal(torch.nan_to_num(a, 5.0, 6.0, 7.0), torch.nan_to_num(b, 5.0, 6.0, 7.0))
        out, norm = msr.msr_clip_gradients(g, 1.0, out=[torch.empty_like(t) for t in g])
        assert not np.isfinite(float(norm)) and all(same(a, b) for a, b in zip(out, ref))
        out, norm = msr.msr_clip_gradients(g, 1.0)
        assert not np.isfinite(float(norm)) and all(same(a, b) for a, b in zip(out, ref))
    over = [torch.full((9000,), 3e38, device=dev)]  # finite, its norm is not
    out, norm = msr.msr_clip_gradients([over[0].clone()], 1.0)
    assert float(norm) == float("inf") and torch.equal(out[0], over[0])


def test_iterables_and_the_same_tensor_twice():
    torch, dev = torch_dev()
    msr = _msr()
    g = [torch.randn(1000, device=dev), torch.randn(30, device=dev).bfloat16()]
    want, norm = msr.msr_clip_gradients(g, 0.25, out=[torch.empty_like(t) for t in g])
    out, n2 = msr.msr_clip_gradients(iter(g), 0.25, out=(torch.empty_like(t) for t in g))
    assert torch.equal(norm, n2) and len(out) == 2 and all(torch.equal(a, b) for a, b in zip(out, want))
    # for the norm a tensor may be there twice, also read for two outputs, but not scaled twice in place
    both = msr.msr_gradient_norm([g[0], g[0]])
    assert abs(float(both) - 2 ** 0.5 * float(g[0].double().norm())) <= 1e-6 * float(both)
    out, _ = msr.msr_clip_gradients([g[0], g[0]], 0.25, out=[torch.empty_like(g[0]) for _ in range(2)])
    assert torch.equal(out[0], out[1])
    for args in (dict(), dict(out=[out[0], out[0]]), dict(out=[g[0], out[1]]), dict(out=[out[0], g[0]])):
        with pytest.raises(msr.MsrError, match="overlaps"):
            msr.msr_clip_gradients([g[0], g[0]], 0.25, **args)


def test_more_than_two_to_the_31_elements():
    torch, dev = torch_dev()
    msr = _msr()
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g[-3:] = 2.0
    g[0] = 1.0
    out, norm = msr.msr_clip_gradients([g], 1.0)
    assert abs(float(norm) - 13 ** 0.5) < 1e-6
    assert float(out[0][-1]) == float(torch.tensor(2 / 13 ** 0.5).bfloat16()) and float(out[0][1]) == 0
    del g, out


def test_in_a_graph_and_on_two_streams():
    torch, dev = torch_dev()
    msr = _msr()
    sizes = [(30000, "f32"), (777, "bf16"), (100001, "bf16")]
    sets = [make(torch, dev, sizes, seed=i)[0] for i in range(3)]
    eager = [msr.msr_clip_gradients(g, 0.5, out=[torch.empty_like(t) for t in g]) for g in sets]
    live = [t.clone() for t in sets[0]]
    msr.msr_clip_gradients(live, 0.5, out=[torch.empty_like(t) for t in live])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, norm = msr.msr_clip_gradients(live, 0.5, out=[torch.empty_like(t) for t in live])
    for i in (1, 2, 0, 1):
        for t, s in zip(live, sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, eager[i][1]) and all(torch.equal(a, b) for a, b in zip(out, eager[i][0]))
        msr.msr_gradient_norm(sets[0])
    streams = [torch.cuda.Stream() for _ in sets]
    got = [msr.msr_clip_gradients(g, 0.5, out=[torch.empty_like(t) for t in g], stream=s) for g, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for (a, n), (b, m) in zip(got, eager):
        assert torch.equal(n, m) and all(torch.equal(u, v) for u, v in zip(a, b))
