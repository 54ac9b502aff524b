"""copy_slots, free_slots and compact_slots against plain indexing on copies of the pools: every bit of
every pool row, the rows that no pair names among them."""
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200.synth import Dims

pytestmark = pytest.mark.gpu
SMALL = Dims(num_k_heads=1, num_v_heads=1)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


def _pools(P, dims, dev, seed=1):
    """Random bits, NaN and infinities among them; compared as integers."""
    g = torch.Generator(device=dev).manual_seed(seed)
    draw = lambda shape: torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device=dev, dtype=torch.int64) \
        .to(torch.int32).view(torch.float32)
    return draw((P, dims.num_v_heads, 128, 128)), draw((P, 3, dims.conv_channels))


def _same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


def _copied(pool, src, dst):
    new = pool.clone()
    for s, d in zip(src, dst):
        new[d] = pool[s] if s >= 0 else 0
    return new


def _check_copy(P, src, dst, dims, dev):
    st, cv = _pools(P, dims, dev, seed=P + len(src))
    want = [_copied(p, src, dst) for p in (st, cv)]
    gdn.copy_slots(src, dst, st, cv, dims=dims)
    torch.cuda.synchronize(dev)
    assert _same(st, want[0]) and _same(cv, want[1])
    assert gdn.last_device_error() == 0


@pytest.mark.parametrize("P,src,dst", [
    (2, [0], [1]),                              # a copy
    (9, [4] * 8, [0, 1, 2, 3, 5, 6, 7, 8]),     # a fork over the whole pool
    (2, [1, 0], [0, 1]),                        # a swap
    (5, [1, 2, 3, 4, 0], [0, 1, 2, 3, 4]),      # a cycle
    (6, [0, 0, 1, 1, 2, 5], [0, 1, 2, 3, 4, 5]),  # beams: kept, forked, overwritten
    (7, [3, 3, 3], [3, 5, 0]),                  # a row kept and forked
    (4, [-1, 2], [2, 0]),                       # a row moved away and cleared
    (4, [-1, -1, -1, -1], [3, 0, 1, 2]),        # all cleared
    (3, [0, 1, 2], [0, 1, 2]),                  # nothing moves
])
def test_copy_patterns(dev, P, src, dst):
    _check_copy(P, src, dst, SMALL, dev)
    _check_copy(P, src, dst, Dims(num_k_heads=3, num_v_heads=9), dev)


@pytest.mark.parametrize("dims", [SMALL, Dims(num_k_heads=2, num_v_heads=16)])
@pytest.mark.parametrize("P", [1, 2, 17, 40])
def test_copy_random(dev, P, dims):
    for seed in range(6):
        g = torch.Generator().manual_seed(100 * P + seed)
        n = int(torch.randint(0, P + 1, (1,), generator=g))
        dst = torch.randperm(P, generator=g)[:n].tolist()
        src = torch.randint(-1, P, (n,), generator=g).tolist()
        _check_copy(P, src, dst, dims, dev)


def test_copy_model_shape(dev):
    """The 27B layer's rows: forks, a swap, a clear, rows left alone; tables as tensors."""
    st, cv = _pools(12, gdn.MODEL, dev)
    src, dst = [0, 0, 3, 4, -1, 11], [7, 9, 4, 3, 5, 6]
    want = [_copied(p, src, dst) for p in (st, cv)]
    gdn.copy_slots(torch.tensor(src, dtype=torch.int32, device=dev), torch.tensor(dst), st, cv)
    torch.cuda.synchronize(dev)
    assert _same(st, want[0]) and _same(cv, want[1])


def test_copy_large_sets(dev):
    """One cycle of 512 rows (the largest set that overwrites its sources), a fork into 1100 rows (several
    launches), 700 separate swaps (several launches); a cycle of 513 is refused."""
    P = 1500
    _check_copy(P, [(i + 1) % 512 for i in range(512)], list(range(512)), SMALL, dev)
    _check_copy(P, [1400] * 1100, list(range(1100)), SMALL, dev)
    _check_copy(P, [i ^ 1 for i in range(1400)], list(range(1400)), SMALL, dev)
    st, cv = _pools(513, SMALL, dev)
    before = st.clone()
    with pytest.raises(gdn.GdnError):
        gdn.copy_slots([(i + 1) % 513 for i in range(513)], list(range(513)), st, cv, dims=SMALL)
    torch.cuda.synchronize(dev)
    assert _same(st, before)


def test_free_slots(dev):
    st, cv = _pools(6, SMALL, dev)
    want = [_copied(p, [-1, -1], [1, 4]) for p in (st, cv)]
    gdn.free_slots([1, 4], st, cv, dims=SMALL)
    gdn.free_slots([], st, cv, dims=SMALL)
    torch.cuda.synchronize(dev)
    assert _same(st, want[0]) and _same(cv, want[1])


@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("P", [1, 2, 5, 33, 64])
def test_compact(dev, P, clear):
    for seed, share in enumerate((0.0, 0.3, 0.6, 1.0)):
        g = torch.Generator().manual_seed(10 * P + seed)
        live = (torch.rand(P, generator=g) < share).tolist()
        st, cv = _pools(P, SMALL, dev, seed=seed)
        before = [st.clone(), cv.clone()]
        remap = gdn.compact_slots(live if seed % 2 else torch.tensor(live, device=dev), st, cv, clear=clear, dims=SMALL)
        torch.cuda.synchronize(dev)
        n = sum(live)
        assert remap.dtype == torch.int32 and tuple(remap.shape) == (P,)
        assert sorted(int(r) for r in remap if r >= 0) == list(range(n))
        for old, new in zip(before, (st, cv)):
            for i in range(P):
                assert (int(remap[i]) >= 0) == live[i]
                if live[i]:
                    assert _same(new[int(remap[i])], old[i])
                    if i < n:
                        assert int(remap[i]) == i
            for i in range(n, P):
                assert _same(new[i], torch.zeros_like(old[i]) if clear else old[i])


def test_graph_and_streams(dev):
    """A captured copy keeps its tables when the host lists are gone, and two copies on two streams work
    on their own pools."""
    st, cv = _pools(5, SMALL, dev)
    st2, cv2 = _pools(5, SMALL, dev, seed=9)
    src, dst = [1, 2, 0, 0], [0, 1, 2, 4]
    want, want2 = [st, cv], [st2, cv2]
    for _ in range(3):
        want = [_copied(p, src, dst) for p in want]
        want2 = [_copied(p, src, dst) for p in want2]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        gdn.copy_slots(list(src), list(dst), st, cv, dims=SMALL)
    for _ in range(3):
        with torch.cuda.stream(s1):
            graph.replay()
        with torch.cuda.stream(s2):
            gdn.copy_slots(src, dst, st2, cv2, dims=SMALL)
    torch.cuda.synchronize(dev)
    assert _same(st, want[0]) and _same(cv, want[1])
    assert _same(st2, want2[0]) and _same(cv2, want2[1])


def test_refusals(dev):
    st, cv = _pools(4, SMALL, dev)
    before = [st.clone(), cv.clone()]
    for src, dst in (([0, 1], [2, 2]), ([4], [0]), ([-2], [0]), ([0], [4]), ([0], [-1])):
        with pytest.raises(gdn.GdnError):
            gdn.copy_slots(src, dst, st, cv, dims=SMALL)
    with pytest.raises(ValueError):
        gdn.copy_slots([0, 1], [2], st, cv, dims=SMALL)
    with pytest.raises(ValueError):
        gdn.copy_slots([2 ** 31], [0], st, cv, dims=SMALL)
    with pytest.raises(TypeError):
        gdn.copy_slots(torch.tensor([0.0]), [1], st, cv, dims=SMALL)
    with pytest.raises(ValueError):
        gdn.copy_slots([0], [1], st, cv[:3], dims=SMALL)
    with pytest.raises(ValueError):
        gdn.copy_slots([0], [1], st, cv)  # the pools of other dims
    with pytest.raises(ValueError):
        gdn.compact_slots([True] * 3, st, cv, dims=SMALL)
    with pytest.raises(ValueError):
        gdn.compact_slots(torch.ones((4, 1)), st, cv, dims=SMALL)
    torch.cuda.synchronize(dev)
    assert _same(st, before[0]) and _same(cv, before[1])
