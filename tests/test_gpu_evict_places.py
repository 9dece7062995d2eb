"""Where an eviction may put keys and values: destinations that lie in one allocation without
sharing an element are served, destinations that share one are refused."""
import pytest

from tests.test_gpu_evict import INVALID_ARGUMENT, Case

pytestmark = pytest.mark.gpu

PAGE = 64


def _into(k_to, v_to):
    """A case whose fresh pages are these (another pool), filled with what a check compares."""
    c = Case([300, 100, 131, 500], 130, 2, 20, hk=2, dim=64, spare=1)
    c.k_to, c.v_to = k_to, v_to
    k_to.normal_()
    v_to.normal_()
    c.to_before = (k_to.clone(), v_to.clone())
    return c


def _flat(n):
    import torch
    return torch.zeros(n, dtype=torch.bfloat16, device="cuda")


def _pages():
    return Case([300, 100, 131, 500], 130, 2, 20, hk=2, dim=64, spare=1).k_to.shape[0]


@pytest.mark.parametrize("kind", ["joint", "joint, keys behind values", "slot by slot", "head by head", "values the other way round",
                                  "halves of a wide head", "one behind the other", "every other page"])
def test_destinations_that_share_no_element(kind):
    N = _pages()
    if kind.startswith("joint"):
        both = _flat(N * 2 * PAGE * 2 * 64).view(N, 2, PAGE, 2, 64)
        k, v = both[:, 0], both[:, 1]
        if kind != "joint":
            k, v = v, k
    elif kind == "slot by slot":
        both = _flat(N * PAGE * 2 * 2 * 64).view(N, PAGE, 2, 2, 64)
        k, v = both[:, :, 0], both[:, :, 1]
    elif kind == "head by head":
        both = _flat(N * 2 * 2 * PAGE * 64).view(N, 2, 2, PAGE, 64)
        k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    elif kind == "values the other way round":
        both = _flat(N * 2 * PAGE * 2 * 64).view(N, 2, PAGE * 2 * 64)
        k, v = both[:, 0].view(N, PAGE, 2, 64), both[:, 1].view(N, 2, PAGE, 64).transpose(1, 2)
    elif kind == "halves of a wide head":
        both = _flat(N * PAGE * 2 * 128).view(N, PAGE, 2, 128)
        k, v = both[..., :64], both[..., 64:]
    elif kind == "one behind the other":
        both = _flat(2 * N * PAGE * 2 * 64).view(2, N, PAGE, 2, 64)
        k, v = both[1], both[0]
    else:
        both = _flat(2 * N * PAGE * 2 * 64).view(2 * N, PAGE, 2, 64)
        k, v = both[::2], both[1::2]
    c = _into(k, v)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("pool", ["other", "same"])
def test_views_of_a_latent_cache(pool):
    """Keys and values that share elements of every position, in the caches and in the fresh pages alike."""
    import torch
    c = Case([300, 100, 131, 500], 130, 2, 20, hk=2, dim=64, spare=1, pool=pool)
    views = lambda t: (t[..., :64], t[..., 32:])
    src = torch.randn(c.k.shape[0], PAGE, 2, 96, device="cuda").to(torch.bfloat16)
    dst = src if pool == "same" else torch.randn(c.k_to.shape[0], PAGE, 2, 96, device="cuda").to(torch.bfloat16)
    (c.k, c.v), (c.k_to, c.v_to) = views(src), views(dst)
    c.before, c.to_before = (c.k.clone(), c.v.clone()), (c.k_to.clone(), c.v_to.clone())
    assert c.run() == 0
    c.check()
    if pool == "other":      # one slot further in the fresh pages only
        room = torch.zeros(dst.numel() + 1024, dtype=torch.bfloat16, device="cuda")
        c.k_to = room.as_strided(c.k_to.shape, c.k_to.stride(), 0)
        c.v_to = room.as_strided(c.k_to.shape, c.k_to.stride(), 2 * 96 + 32)
        assert c.run() == INVALID_ARGUMENT and bool((room == 0).all())


@pytest.mark.parametrize("kind", ["a page apart", "a slot apart", "half a page apart", "half a head apart", "joint, a page apart",
                                  "the other way round, a page apart", "other page strides"])
def test_destinations_that_share_elements(kind):
    import torch
    N, page = _pages(), PAGE * 2 * 64
    room = _flat((2 * N + 2) * page)
    at = lambda off, strides=(page, 128, 64, 1): room.as_strided((N, PAGE, 2, 64), strides, off)
    if kind == "a page apart":
        k, v = at(0), at(page)
    elif kind == "a slot apart":
        k, v = at(128), at(0)
    elif kind == "half a page apart":
        k, v = at(0), at(page // 2)
    elif kind == "half a head apart":
        k, v = at(32), at(0)
    elif kind == "joint, a page apart":      # keys of one page on values of the next
        k, v = at(0, (2 * page, 128, 64, 1)), at(page * 3 // 2, (2 * page, 128, 64, 1))
    elif kind == "the other way round, a page apart":
        k, v = at(0), at(page, (page, 64, 64 * PAGE, 1))
    else:
        k, v = at(0), at(page, (2 * page, 128, 64, 1))
    c = _into(k, v)
    before = room.clone()
    assert c.run() == INVALID_ARGUMENT
    assert bool((c.keep == 7).all()) and bool((c.new_len == 7).all()) and torch.equal(room, before)
